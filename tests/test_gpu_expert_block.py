"""examples/expert_block.py, the int8, grouped and head-norm operators in one
block, against the same block in float64 from the dequantized weights.

Tolerance (relative Frobenius norm, fixed before the first run): the two sides
differ by bf16 roundings (2^-9 relative each, at most five in a row) and by the
quantized codes that those roundings move to a neighbour.  A code of step d
(relative to its value) moves with probability 2^-9 / d and by d, an rms of
sqrt(2^-9 d): 0.7 % for int8 (d about 1/40), 2.5 % for E2M1 (d about 0.3), and
both halves of a half-block quantize twice.  3 % and 8 %.
"""
import importlib.util
import os

import pytest
import torch

import fp8_quantized_linear_mxq_amd as mxq

pytestmark = pytest.mark.gpu

_path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_block.py")
_spec = importlib.util.spec_from_file_location("expert_block", _path)
eb = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(eb)

E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def dense(q):
    """A quantized operand in float64 on the host."""
    if q.fmt == mxq.BF16:
        return q.codes.double().cpu()
    if q.fmt == mxq.INT8:
        return q.codes.view(torch.int8)[:, :q.cols].double().cpu() * q.scales.double().cpu().view(-1, 1)
    b = q.codes[:, :q.cols // 2].cpu().long()
    v = E2M1[torch.stack([b & 15, b >> 4], 2).view(q.rows, q.cols)]
    s = torch.exp2(q.scales[:, :q.cols // 32].cpu().double() - 127)
    return v * s.repeat_interleave(32, 1)


def coded(x, fmt):
    """x (float64) as its quantized values; the framework's own quantize, whose codes are tested elsewhere."""
    x = x.bfloat16().cuda()
    return dense(mxq.bf16_operand(x) if fmt == mxq.BF16 else mxq.quantize(x, fmt))


def head_norm(x, gain, cos, sin):
    n = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * gain
    a, b = n.chunk(2, -1)
    c, s = cos[:, None], sin[:, None]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def close(got, want, base, tol):
    """The update got - base against want - base."""
    got, want = got.double().cpu() - base, want - base
    assert torch.isfinite(got).all()
    assert (got - want).norm() <= tol * want.norm(), float((got - want).norm() / want.norm())


@pytest.mark.parametrize("tokens", [1, 7, 130])
@pytest.mark.parametrize("pair,tol", [("int8", 0.03), ("mxfp4", 0.08), ("w4a16", 0.03)])
def test_block(pair, tol, tokens):
    blk = eb.ExpertBlock(width=256, heads=4, kv_heads=2, head_dim=64, experts=9, topk=2, hidden=128,
                         pair=pair, n_pos=512, seed=tokens)
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    x = torch.randn(tokens, 256, generator=gen, device="cuda").bfloat16()
    pos = torch.arange(5, 5 + tokens, dtype=torch.int32, device="cuda")
    h = blk.attention(x, pos)
    p, pick = blk.route(h)
    y = blk.experts(h, p, pick)

    # attention half
    xd = x.double().cpu()
    qkv = coded(xd, mxq.INT8) @ dense(blk.wqkv).t()
    q, k, v = qkv.view(tokens, 8, 64).split([4, 2, 2], 1)
    cos, sin = blk.cos.double().cpu()[pos.cpu().long()], blk.sin.double().cpu()[pos.cpu().long()]
    o = eb.causal(head_norm(q, blk.q_gain.double().cpu(), cos, sin),
                  head_norm(k, blk.k_gain.double().cpu(), cos, sin), v)
    close(h, xd + coded(o, mxq.INT8) @ dense(blk.wout).t(), xd, tol)

    # expert half, from the h that was computed
    hd, pd, pick = h.double().cpu(), p.double().cpu(), pick.cpu()
    w_up, w_down = dense(blk.w_up).view(9, 256, 256), dense(blk.w_down).view(9, 256, 128)
    ha = coded(hd, blk.act)
    want = hd.clone()
    for t in range(tokens):
        for j in range(2):
            up = w_up[pick[t, j]] @ ha[t]
            act = up[:128] / (1 + torch.exp(-up[:128])) * up[128:]
            want[t] += pd[t, j] * (w_down[pick[t, j]] @ coded(act[None], blk.act)[0])
    close(y, want, hd, tol)


def test_a_sequence_split_in_two_calls_routes_alike():
    """Experts see rows, not sequences: a token's output does not depend on the others."""
    blk = eb.ExpertBlock(width=256, heads=4, kv_heads=2, head_dim=64, experts=9, topk=2, hidden=128)
    h = torch.randn(40, 256, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").bfloat16()
    p, pick = blk.route(h)
    whole = blk.experts(h, p, pick)
    for lo, hi in ((0, 1), (1, 40)):
        part = blk.experts(h[lo:hi], p[lo:hi], pick[lo:hi])
        # int8 sums are exact, so the split changes nothing
        assert torch.equal(part, whole[lo:hi])
