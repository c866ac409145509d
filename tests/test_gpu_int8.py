"""GPU parity of the row-wise int8 quantize and the int8 x int8 GEMM against
the float64 oracle: codes and scales bit for bit, outputs within the bound of
every GEMM route (the integer sum is exact, so only the two scale products,
the epilogue and the bf16 rounding differ)."""
import numpy as np
import pytest

from fp8_quantized_linear_mxq_amd import workloads as wl
from oracle import hadamard as oh
from oracle import int8 as o8
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


def _draw(rng, rows, cols, dtype):
    x = rng.standard_t(3, size=(rows, cols)) * np.exp(rng.uniform(-5, 5, size=cols))
    x = x.astype(np.float32)
    return wl.f32_to_bf16_bits(x) if dtype == "bf16" else x


def _operand(q, s):
    import torch
    import fp8_quantized_linear_mxq_amd as mxq
    return mxq.int8_operand(torch.from_numpy(q).cuda(), torch.from_numpy(np.asarray(s, np.float32)).cuda())


def _check_codes(got, vals, tag):
    q, s = o8.quantize(vals)
    assert np.array_equal(got.scales.cpu().numpy().ravel(), s), f"{tag}: scales"
    codes = got.codes.cpu().numpy().view(np.int8)
    assert np.array_equal(codes, q), f"{tag}: {np.sum(codes != q)} codes differ"


# one wave per row (up to 2048 columns: 1 .. 4 pieces), a workgroup per row (2 ..
# 16 pieces), and rows too long to hold in registers
QSHAPES = [(1, 32), (3, 1152), (5, 4128), (1, 8160), (2, 16384), (3, 16416), (2049, 96), (2050, 1152),
           (2048, 2400), (2051, 4096), (7, 640), (6, 2048), (4, 2080), (3, 11264), (2, 24608), (2, 32768),
           (3, 32800)]


@pytest.mark.parametrize("rows,cols", QSHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize(rows, cols, dtype):
    import fp8_quantized_linear_mxq_amd as mxq
    gu.say(f"int8 quantize {rows}x{cols} {dtype}")
    x = _draw(np.random.default_rng(rows + cols), rows, cols, dtype)
    got = mxq.quantize(gu.act_to_dev(x, dtype), mxq.INT8)
    _check_codes(got, gu.act_values(x, dtype), f"{rows}x{cols}")


@pytest.mark.parametrize("rows,cols", [(3, 128), (7, 1152), (2, 16512), (2049, 1536), (5, 512), (3, 3200), (2, 8192), (3, 12288)])
@pytest.mark.parametrize("had", [16, 32, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_rotated(rows, cols, had, dtype):
    import fp8_quantized_linear_mxq_amd as mxq
    gu.say(f"int8 quantize {rows}x{cols} {dtype} rotated by {had}")
    rng = np.random.default_rng(had + cols)
    x = (rng.standard_t(4, size=(rows, cols))).astype(np.float32)
    # short mantissas: the rotation's sums stay exact (the documented domain)
    x = wl.bf16_to_f32(wl.f32_to_bf16_bits(x))
    dev = gu.to_dev_bf16(wl.f32_to_bf16_bits(x)) if dtype == "bf16" else gu.to_dev_f32(x)
    got = mxq.quantize(dev, mxq.INT8, hadamard=had)
    _check_codes(got, oh.rotate(x, had, 7), f"rotated {had}")


def test_quantize_ties_zeros_and_small_rows():
    """Exact halves (to even), quotients next to halves, zero rows, rows whose
    scale is subnormal or underflows to zero, and the largest finite values."""
    import fp8_quantized_linear_mxq_amd as mxq
    rng = np.random.default_rng(9)
    k = 512
    x = np.zeros((12, k), np.float32)
    half = (np.arange(k) % 254 - 126.5).astype(np.float32)
    for r in range(4):                                  # scale 2**(3r - 4) exactly
        x[r] = half * np.float32(2.0 ** (3 * r - 4))
        x[r, 0] = 127 * np.float32(2.0 ** (3 * r - 4))
    for r in range(4, 7):                               # neighbours of halves under odd scales
        s = np.float32(rng.uniform(0.5, 2))
        x[r] = (half.astype(np.float64) * np.float64(s)).astype(np.float32)
        x[r] = np.nextafter(x[r], np.float32(np.inf) if r % 2 else np.float32(-np.inf))
        x[r, 0] = np.float32(127.0 * float(s))
    x[8] = rng.standard_normal(k).astype(np.float32) * np.float32(1e-38)
    x[9] = rng.standard_normal(k).astype(np.float32) * np.float32(3e-43)
    x[10, 5] = np.float32(1e-45)
    x[11] = rng.standard_normal(k).astype(np.float32) * np.float32(8e37)
    gu.say("int8 quantize ties, zero and small rows")
    _check_codes(mxq.quantize(gu.to_dev_f32(x), mxq.INT8), x, "edges")


def test_quantize_strides_outputs_and_streams():
    """Rows wider than K in and out, an odd row count, guard bytes around the
    codes, a stream of its own, an empty input."""
    import torch
    import fp8_quantized_linear_mxq_amd as mxq
    gu.say("int8 quantize strided, on its own stream")
    rng = np.random.default_rng(3)
    x = _draw(rng, 33, 192, "bf16")
    xd = gu.to_dev_bf16(x)[:, :160]
    codes = torch.full((33, 208), 77, dtype=torch.uint8, device="cuda")
    scales = torch.full((33, 4), -1.0, dtype=torch.float32, device="cuda")
    out = mxq.QTensor(mxq.INT8, 33, 160, codes, scales)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    mxq.quantize(xd, mxq.INT8, out=out, stream=st)
    st.synchronize()
    q, s = o8.quantize(wl.bf16_to_f32(x)[:, :160])
    c = codes.cpu().numpy()
    assert np.array_equal(c[:, :160].view(np.int8), q) and np.all(c[:, 160:] == 77)
    sc = scales.cpu().numpy()
    assert np.array_equal(sc[:, 0], s) and np.all(sc[:, 1:] == -1)
    e = mxq.quantize(torch.empty((0, 64), device="cuda"), mxq.INT8)
    assert e.codes.shape[0] == 0


def test_quantize_lowrank_and_noalloc():
    import ctypes as C
    import torch
    import fp8_quantized_linear_mxq_amd as mxq
    from fp8_quantized_linear_mxq_amd import _lib
    gu.say("int8 quantize with the low-rank projection, allocation-free call")
    rng = np.random.default_rng(2)
    m, k, r = 37, 256, 32
    x = _draw(rng, m, k, "bf16")
    l1 = wl.f32_to_bf16_bits(rng.normal(0, 0.02, (r, k)).astype(np.float32))
    u = torch.empty((m, r), dtype=torch.float32, device="cuda")
    xd = gu.to_dev_bf16(x)
    got = mxq.quantize(xd, mxq.INT8, l1t=gu.to_dev_bf16(l1), u=u)
    xv, lv = wl.bf16_to_f32(x).astype(np.float64), wl.bf16_to_f32(l1).astype(np.float64).T
    _check_codes(got, wl.bf16_to_f32(x), "low rank")
    assert np.all(np.abs(u.cpu().numpy() - xv @ lv) <= 1e-5 * (np.abs(xv) @ np.abs(lv)))
    out = mxq.empty_qtensor(mxq.INT8, m, k)
    oc = out.c()
    st = mxq.load().mxq_quantize_noalloc(C.c_void_p(xd.data_ptr()), 2, m, k, k, 0, None, None, 0, None, 0,
                                         C.byref(oc), _lib._stream(None))
    assert st == 0
    _check_codes(out, wl.bf16_to_f32(x), "noalloc")


def test_quantize_debug_checks(monkeypatch):
    import torch
    import fp8_quantized_linear_mxq_amd as mxq
    gu.say("int8 quantize debug checks")
    monkeypatch.setenv("MXQ_DEBUG_CHECKS", "1")
    x = torch.ones((4, 64), device="cuda")
    mxq.quantize(x, mxq.INT8)
    x[2, 5] = float("nan")
    mxq.quantize(x, mxq.INT8)
    with pytest.raises(mxq.MxqError) as ei:
        mxq.quantize(torch.ones((4, 64), device="cuda"), mxq.INT8)
    assert ei.value.status == 8
    mxq.quantize(torch.ones((4, 64), device="cuda"), mxq.INT8)


def _codes(rng, rows, cols):
    q = np.clip(np.rint(rng.standard_normal((rows, cols)) * 40), -127, 127).astype(np.int8)
    return q, np.exp(rng.uniform(-6, 2, rows)).astype(np.float32)


# few rows (one and two 16-row tiles), each workgroup tile, ragged everywhere,
# K that ends inside a K-tile and a step
GSHAPES = [(1, 1, 32), (1, 4608, 1152), (3, 100, 96), (16, 33, 2080), (17, 513, 160), (32, 64, 4096),
           (33, 65, 32), (100, 130, 224), (130, 250, 384), (1500, 1400, 288), (777, 1001, 1184),
           (2300, 4000, 416), (4100, 3900, 160)]


@pytest.mark.parametrize("m,n,k", GSHAPES)
def test_gemm(m, n, k):
    import fp8_quantized_linear_mxq_amd as mxq
    gu.say(f"int8 gemm {m}x{n}x{k}")
    rng = np.random.default_rng(m + n + k)
    (qa, sa), (qw, sw) = _codes(rng, m, k), _codes(rng, n, k)
    y = mxq.gemm(_operand(qa, sa), _operand(qw, sw))
    r = gu.check_gemm(y, o8.dequantize(qa, sa), o8.dequantize(qw, sw), 1.0, tag=f"int8 {m}x{n}x{k}")
    gu.say(f"  worst err/tol {r:.3g}")


@pytest.mark.parametrize("m", [5, 40, 300])
def test_gemm_bias_lowrank_colmap_strided(m):
    import torch
    import fp8_quantized_linear_mxq_amd as mxq
    gu.say(f"int8 gemm M={m} with bias, low-rank branch, column map, strides")
    n, k, r, n_out = 200, 352, 32, 215
    rng = np.random.default_rng(m)
    (qa, sa), (qw, sw) = _codes(rng, m, k), _codes(rng, n, k)
    u = (rng.standard_normal((m, r)) * 4).astype(np.float32)
    l2 = wl.bf16_to_f32(wl.f32_to_bf16_bits(rng.normal(0, 0.02, (r, n_out)).astype(np.float32)))
    bias = wl.bf16_to_f32(wl.f32_to_bf16_bits(rng.normal(0, 1, n_out).astype(np.float32)))
    perm = rng.permutation(n_out)[:n].astype(np.int32)
    wide = torch.zeros((m, k + 48), dtype=torch.int8, device="cuda")
    wide[:, :k] = torch.from_numpy(qa).cuda()
    wsc = torch.zeros((n, 3), dtype=torch.float32, device="cuda")
    wsc[:, 0] = torch.from_numpy(sw).cuda()
    a = mxq.int8_operand(wide[:, :k], torch.from_numpy(sa).cuda())
    w = mxq.QTensor(mxq.INT8, n, k, torch.from_numpy(qw).cuda(), wsc)
    args = dict(u=gu.to_dev_f32(u), l2t=gu.to_dev_bf16(wl.f32_to_bf16_bits(np.ascontiguousarray(l2.T))),
                bias=gu.to_dev_bf16(wl.f32_to_bf16_bits(bias)))
    ad, wd = o8.dequantize(qa, sa), o8.dequantize(qw, sw)
    x1 = np.abs(u).astype(np.float64)                  # S counts |u| |L2|
    ext = dict(u=u.astype(np.float64), x=x1, l1=np.eye(r))
    out = torch.full((m, n_out + 9), -7.0, dtype=torch.bfloat16, device="cuda")
    y = mxq.gemm(a, w, n_out=n_out, w_out_col=torch.from_numpy(perm).cuda(), out=out, **args)
    got = y.float().cpu().numpy()
    rest = np.setdiff1d(np.arange(n_out + 9), perm)
    assert np.all(got[:, rest] == -7.0)
    gu.check_gemm(y, ad, wd, 1.0, l2=l2[:, perm], bias=bias[perm], cols=perm, tag="colmap", **ext)
    # no map, aligned rows: the staged stores
    y = mxq.gemm(a, w, **dict(args, l2t=args["l2t"][:n].contiguous(), bias=args["bias"][:n].contiguous()))
    gu.check_gemm(y, ad, wd, 1.0, l2=l2[:, :n], bias=bias[:n], tag="plain", **ext)
    # the same rows as two weight groups
    y = mxq.gemm_mixed(a, [mxq.QTensor(mxq.INT8, 70, k, w.codes[:70], wsc[:70]),
                           mxq.QTensor(mxq.INT8, n - 70, k, w.codes[70:], wsc[70:])],
                       torch.from_numpy(perm).cuda(), n_out, **args)
    gu.check_gemm(y, ad, wd, 1.0, l2=l2[:, perm], bias=bias[perm], cols=perm, tag="mixed", **ext)


@pytest.mark.parametrize("m", [2, 70, 600])
def test_gemm_sum_is_exact(m):
    """Unit scales and codes of -1, 0, 1: every output is a small integer that
    bf16 holds, so nothing may be off by even one; and the longest K with the
    largest codes, whose sum only just stays within int32."""
    import torch
    import fp8_quantized_linear_mxq_amd as mxq
    gu.say(f"int8 gemm exact sums M={m}")
    rng = np.random.default_rng(m)
    n, k = 150, 256
    qa = rng.integers(-1, 2, (m, k)).astype(np.int8)
    qw = rng.integers(-1, 2, (n, k)).astype(np.int8)
    y = mxq.gemm(_operand(qa, np.ones(m)), _operand(qw, np.ones(n))).float().cpu().numpy()
    assert np.array_equal(y, (qa.astype(np.int64) @ qw.astype(np.int64).T).astype(np.float32))
    k = 1 << 17
    one = torch.full((m, k), 127, dtype=torch.int8, device="cuda")
    w = torch.full((20, k), 127, dtype=torch.int8, device="cuda")
    w[7] = -127
    s = torch.ones(m, device="cuda")
    y = mxq.gemm(mxq.int8_operand(one, s), mxq.int8_operand(w, torch.ones(20, device="cuda"))).double().cpu()
    want = torch.tensor(float(127 * 127 * k)).to(torch.bfloat16).double()
    assert torch.all(y[:, 7] == -want) and torch.all(y[:, 8:] == want) and torch.all(y[:, :7] == want)


def test_layer_on_other_stream_and_in_a_graph():
    """quantize + gemm captured in a HIP graph, replayed several times with new
    inputs and eager work between, each replay against the eager result."""
    import torch
    import fp8_quantized_linear_mxq_amd as mxq
    gu.say("int8 layer in a graph")
    rng = np.random.default_rng(1)
    qw, sw = _codes(rng, 300, 256)
    w = _operand(qw, sw)
    for m in (4, 200):
        x = torch.randn((m, 256), device="cuda").to(torch.bfloat16)
        q = mxq.empty_qtensor(mxq.INT8, m, 256)
        y = torch.empty((m, 300), dtype=torch.bfloat16, device="cuda")
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            mxq.gemm(mxq.quantize(x, mxq.INT8, out=q), w, out=y)
        torch.cuda.current_stream().wait_stream(st)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mxq.gemm(mxq.quantize(x, mxq.INT8, out=q), w, out=y)
        for i in range(4):
            x.copy_(torch.randn((m, 256), device="cuda") * (i + 1))
            g.replay()
            torch.cuda.synchronize()
            eager = mxq.gemm(mxq.quantize(x, mxq.INT8), w)
            assert torch.equal(y, eager)


# Grids of one or two 64 x 64 tiles per compute unit: every number of K-tiles
# around the four stages, with and without a partial last one.
@pytest.mark.parametrize("k", [32, 128, 160, 256, 384, 512, 544, 640, 768, 992, 1024, 1152, 4128])
def test_gemm_staged_k(k):
    import fp8_quantized_linear_mxq_amd as mxq
    m, n = 200, 770
    gu.say(f"int8 gemm {m}x{n}x{k}")
    rng = np.random.default_rng(k)
    (qa, sa), (qw, sw) = _codes(rng, m, k), _codes(rng, n, k)
    y = mxq.gemm(_operand(qa, sa), _operand(qw, sw))
    gu.check_gemm(y, o8.dequantize(qa, sa), o8.dequantize(qw, sw), 1.0, tag=f"int8 {m}x{n}x{k}")


# small products of more than 16 rows, with one and with two weight tiles per
# workgroup; 512 and just over 512 tiles of 64 x 64
@pytest.mark.parametrize("m,n,k", [(100, 500, 288), (100, 900, 1184), (250, 500, 96), (1024, 2048, 1184),
                                   (1030, 2048, 160), (2000, 1000, 256)])
def test_gemm_small_and_middle(m, n, k):
    test_gemm(m, n, k)


@pytest.mark.parametrize("m,n", [(60, 90), (1000, 2500)])
def test_gemm_lowrank_rows_and_tiles(m, n):
    """The low-rank branch on the staged tiles (one per compute unit) and on
    those of a larger grid."""
    import fp8_quantized_linear_mxq_amd as mxq
    k, r = 160, 16
    gu.say(f"int8 gemm {m}x{n}x{k} with a rank-{r} branch")
    rng = np.random.default_rng(m)
    (qa, sa), (qw, sw) = _codes(rng, m, k), _codes(rng, n, k)
    u = (rng.standard_normal((m, r)) * 4).astype(np.float32)
    l2 = wl.bf16_to_f32(wl.f32_to_bf16_bits(rng.normal(0, 0.02, (r, n)).astype(np.float32)))
    y = mxq.gemm(_operand(qa, sa), _operand(qw, sw), u=gu.to_dev_f32(u),
                 l2t=gu.to_dev_bf16(wl.f32_to_bf16_bits(np.ascontiguousarray(l2.T))))
    gu.check_gemm(y, o8.dequantize(qa, sa), o8.dequantize(qw, sw), 1.0, l2=l2, u=u.astype(np.float64),
                  x=np.abs(u).astype(np.float64), l1=np.eye(r), tag="lowrank")
