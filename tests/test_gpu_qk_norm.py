"""GPU parity of the per-head norm with the position rotation against the
float64 oracle.  Bound: the sum of squares of D <= 512 terms is a chain of 8
products in a lane and at most 6 sums across lanes (14 roundings), the root,
the quotient, two products and the rotation's three roundings stay under 32
fp32 roundings, so |err| <= 2**-19 (|a| + |b|) over the pair, plus the output
rounding (2**-8 |y| + 2**-133 covers bf16; fp32 outputs have none)."""
import numpy as np
import pytest

from fp8_quantized_linear_mxq_amd import workloads as wl
from oracle import heads as ohd
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


def _pair_size(n, rot, interleaved):
    out = np.abs(n).copy()
    if rot:
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
        s = np.abs(n[..., a]) + np.abs(n[..., b])
        out[..., a] = out[..., b] = s
    return out


def _inputs(seed, tokens, width, d, rot, n_pos, dtype, scale=1.0):
    rng = np.random.default_rng(seed)
    x = (rng.standard_t(4, (tokens, width)) * scale).astype(np.float32)
    g = (1 + 0.2 * rng.standard_normal((2, d))).astype(np.float32)
    ang = rng.uniform(-4, 4, (n_pos, rot // 2))
    if dtype == "bf16":
        x, g = wl.f32_to_bf16_bits(x), wl.f32_to_bf16_bits(g)
    return rng, x, g, np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)


def _expect(x, g, cos, sin, pos, hq, hk, d, rot, eps, inter):
    v = x[:, :(hq + hk) * d].reshape(x.shape[0], hq + hk, d).astype(np.float64)
    res = []
    for part, gain in ((v[:, :hq], g[0]), (v[:, hq:], g[1])):
        n = ohd.norm_rope(part, gain, eps=eps)
        y = ohd.norm_rope(part, gain, cos if rot else None, sin, pos, eps, inter)
        res.append((y, _pair_size(n, rot, inter)))
    return res


def _close(got, want, size, dtype, tag):
    got = got.float().cpu().numpy().astype(np.float64)
    tol = 2.0 ** -19 * size + (2.0 ** -8 * np.abs(want) + 2.0 ** -133 if dtype == "bf16" else 2.0 ** -140)
    err = np.abs(got - want)
    assert np.all(err <= tol), f"{tag}: worst err/tol {np.max(err / tol):.3g}"


# tokens, query heads, key heads, D, rotated part
SHAPES = [(1, 16, 16, 72, 72), (1, 1, 0, 8, 8), (5, 3, 1, 64, 64), (7, 15, 2, 128, 128), (3, 0, 5, 128, 96),
          (33, 33, 3, 80, 16), (2, 4, 4, 200, 200), (9, 5, 1, 256, 64), (4, 2, 2, 512, 512), (3, 2, 1, 264, 264),
          (130, 24, 8, 96, 96), (6, 4, 2, 64, 0), (1000, 16, 4, 64, 64)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_qk_norm_rope(shape, inter, dtype):
    import torch
    import fp8_quantized_linear_mxq_amd as mxq
    t, hq, hk, d, rot = shape
    gu.say(f"qk norm {shape} interleaved={inter} {dtype}")
    width = (hq + 2 * hk) * d
    rng, x, g, cos, sin = _inputs(t + d, t, width, d, rot, t + 20, dtype)
    pos = rng.integers(0, t + 20, t).astype(np.int32)
    xd, gd = gu.act_to_dev(x, dtype), gu.act_to_dev(g, dtype)
    tabs = (gu.to_dev_f32(cos), gu.to_dev_f32(sin)) if rot else (None, None)
    q, k = mxq.qk_norm_rope(xd, hq, hk, d, gd[0], gd[1], *tabs, positions=torch.from_numpy(pos).cuda() if rot else None,
                            eps=1e-5, interleaved=inter)
    (wq, sq), (wk, sk) = _expect(gu.act_values(x, dtype), gu.act_values(g, dtype), cos, sin, pos, hq, hk, d, rot,
                                 1e-5, inter)
    _close(q, wq, sq, dtype, "q")
    _close(k, wk, sk, dtype, "k")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layouts_in_place_and_skipped_tokens(dtype):
    """[head][token] outputs, x rows wider than the heads, the norm in place
    (values untouched), no gains, no positions, tokens outside the tables."""
    import torch
    import fp8_quantized_linear_mxq_amd as mxq
    gu.say(f"qk norm layouts {dtype}")
    t, hq, hk, d, rot = 11, 6, 2, 72, 40
    width = (hq + 2 * hk) * d + 16
    rng, x, g, cos, sin = _inputs(3, t, width, d, rot, t, dtype)
    one = np.ones((2, d))
    xv = gu.act_values(x, dtype)
    tc, ts = gu.to_dev_f32(cos), gu.to_dev_f32(sin)
    (wq, sq), (wk, sk) = _expect(xv, one, cos, sin, None, hq, hk, d, rot, 0.0, False)
    xd = gu.act_to_dev(x, dtype)
    tdt = xd.dtype
    qh = torch.empty((hq, t, d), dtype=tdt, device="cuda")
    kh = torch.empty((hk, t + 3, d), dtype=tdt, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    mxq.qk_norm_rope(xd, hq, hk, d, cos=tc, sin=ts, eps=0.0, q_out=qh.transpose(0, 1),
                     k_out=kh[:, :t].transpose(0, 1), stream=st)
    st.synchronize()
    _close(qh.transpose(0, 1), wq, sq, dtype, "q by head")
    _close(kh[:, :t].transpose(0, 1), wk, sk, dtype, "k by head")
    # in place; positions outside [0, n_pos) leave their token as it was
    pos = np.arange(t, dtype=np.int32)
    pos[2], pos[5] = -1, t
    before = xd.clone()
    mxq.qk_norm_rope(xd, hq, hk, d, cos=tc, sin=ts, eps=0.0, positions=torch.from_numpy(pos).cuda(),
                     q_out=xd[:, :hq * d].unflatten(1, (hq, d)),
                     k_out=xd[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d)))
    keep = [i for i in range(t) if i not in (2, 5)]
    assert torch.equal(xd[[2, 5]], before[[2, 5]])
    assert torch.equal(xd[:, (hq + hk) * d:], before[:, (hq + hk) * d:])
    _close(xd[keep][:, :hq * d].unflatten(1, (hq, d)), wq[keep], sq[keep], dtype, "q in place")
    _close(xd[keep][:, hq * d:(hq + hk) * d].unflatten(1, (hk, d)), wk[keep], sk[keep], dtype, "k in place")


def test_large_small_and_zero_heads():
    """Heads of zeros (eps decides), and values whose squares near fp32's ends."""
    import torch
    import fp8_quantized_linear_mxq_amd as mxq
    gu.say("qk norm value ranges")
    for scale in (0.0, 1e-15, 1e15):
        rng, x, g, cos, sin = _inputs(5, 6, 3 * 64, 64, 64, 6, "f32", scale)
        q, k = mxq.qk_norm_rope(gu.to_dev_f32(x), 2, 1, 64, cos=gu.to_dev_f32(cos), sin=gu.to_dev_f32(sin), eps=1e-30)
        (wq, sq), (wk, sk) = _expect(x, np.ones((2, 64)), cos, sin, None, 2, 1, 64, 64, 1e-30, False)
        _close(q, wq, sq, "f32", f"scale {scale}")
        _close(k, wk, sk, "f32", f"scale {scale}")
    e = torch.empty((0, 192), device="cuda")
    q, k = mxq.qk_norm_rope(e, 2, 1, 64)
    assert q.shape == (0, 2, 64)
