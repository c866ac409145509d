"""GPU parity of the products grouped by expert against the float64 oracle:
each group of rows with its own weights, sizes from none to all of the rows."""
import numpy as np
import pytest

from fp8_quantized_linear_mxq_amd import workloads as wl
from oracle import int8 as o8
from oracle import quantize as oq
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

PAIRS = ["INT8", "MXFP4", "BF16"]


def _acts(rng, pair, m, k):
    """(device operand, exact float64 values)"""
    import torch
    import fp8_quantized_linear_mxq_amd as mxq
    x = (rng.standard_t(3, size=(m, k)) * np.exp(rng.uniform(-2, 2, k))).astype(np.float32)
    if pair == "INT8":
        q, s = o8.quantize(x)
        return mxq.int8_operand(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda()), o8.dequantize(q, s)
    if pair == "BF16":
        b = wl.f32_to_bf16_bits(x)
        return mxq.bf16_operand(gu.to_dev_bf16(b)), wl.bf16_to_f32(b).astype(np.float64)
    q = oq.quantize(x, "MXFP4")
    return gu.qtensor_from_oracle(q, m, k), oq.dequantize(q)


def _weights(rng, pair, rows, k):
    import torch
    import fp8_quantized_linear_mxq_amd as mxq
    w = rng.normal(0, 0.02, (rows, k)).astype(np.float32)
    if pair == "INT8":
        q, s = o8.quantize(w)
        return mxq.int8_operand(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda()), o8.dequantize(q, s)
    q = oq.quantize(w, "MXFP4")
    return gu.qtensor_from_oracle(q, rows, k), oq.dequantize(q)


def _offsets(sizes, first=0):
    return np.concatenate([[first], first + np.cumsum(sizes)]).astype(np.int32)


def _check(pair, sizes, n, k, seed, bias=False, first=0, extra=0):
    import torch
    import fp8_quantized_linear_mxq_amd as mxq
    rng = np.random.default_rng(seed)
    off = _offsets(sizes, first)
    e, m = len(sizes), int(off[-1]) + extra
    gu.say(f"grouped {pair} E={e} M={m} N={n} K={k} sizes {list(sizes)[:12]}")
    (a, av), (w, wv) = _acts(rng, pair, m, k), _weights(rng, pair, e * n, k)
    b = wl.f32_to_bf16_bits(rng.standard_normal((e, n)).astype(np.float32)) if bias else None
    out = torch.full((m, n + 5), -7.0, dtype=torch.bfloat16, device="cuda")
    y = mxq.gemm_grouped(a, w, torch.from_numpy(off).cuda(), out=out,
                         bias=gu.to_dev_bf16(b) if bias else None)
    got = y.float().cpu().numpy()
    covered = np.zeros(m, bool)
    for g in range(e):
        rows = np.arange(off[g], off[g + 1])
        covered[rows] = True
        if len(rows):
            gu.check_gemm(y[:, :n], av[rows], wv[g * n:(g + 1) * n], 1.0,
                          bias=wl.bf16_to_f32(b)[g] if bias else None, rows=rows, tag=f"{pair} group {g}")
    assert np.all(got[~covered] == -7.0) and np.all(got[:, n:] == -7.0)
    if not bias:
        # rows of 16-byte aligned stride leave through the staged stores
        y2 = mxq.gemm_grouped(a, w, torch.from_numpy(off).cuda(),
                              out=torch.full((m, (n + 7) // 8 * 8), -7.0, dtype=torch.bfloat16, device="cuda"))
        assert np.array_equal(y2.float().cpu().numpy()[:, :n], got[:, :n])


# (sizes, n, k): single tokens, empty first / last / middle groups, everything
# in one group, sizes around the 16- and 128-row tiles, more groups than a wave
SIZES = [
    ([1], 40, 128), ([0, 0, 1, 0], 33, 256), ([1] * 8, 64, 384), ([0, 5, 0, 0, 16, 17, 1], 130, 256),
    ([33, 0, 31, 0], 129, 640), ([0, 0, 200, 0], 96, 128), ([40] * 5, 250, 512),
    ([127, 128, 129, 0, 1, 255, 300], 264, 256), ([600, 2, 0, 700], 300, 384), ([3, 0] * 70, 24, 128),
    ([0] * 66 + [9, 150, 61], 48, 256), ([300] * 3 + [0] * 61 + [200, 0, 0, 77], 72, 128),
    ([5] * 64, 40, 128), ([5] * 65, 40, 128), ([1000, 1500], 520, 4224),
]


@pytest.mark.parametrize("case", range(len(SIZES)))
@pytest.mark.parametrize("pair", PAIRS)
def test_grouped(pair, case):
    sizes, n, k = SIZES[case]
    _check(pair, sizes, n, k, seed=case, bias=case % 2 == 1)


@pytest.mark.parametrize("pair", PAIRS)
def test_grouped_uncovered_rows(pair):
    """offsets that begin after row 0 and end before the last row."""
    _check(pair, [2, 0, 6], 72, 128, seed=5, first=3, extra=4)
    _check(pair, [100, 0, 160], 136, 256, seed=6, first=37, extra=90)


@pytest.mark.parametrize("k", [32, 96, 160, 2080])
def test_grouped_int8_odd_k(k):
    _check("INT8", [3, 0, 18], 50, k, seed=k)
    _check("INT8", [120, 0, 180], 200, k, seed=k + 1)


@pytest.mark.parametrize("pair", PAIRS)
def test_grouped_no_rows_in_any_group(pair):
    _check(pair, [0, 0, 0], 40, 128, seed=8, extra=50)


@pytest.mark.parametrize("pair", PAIRS)
def test_grouped_offsets_out_of_range(pair):
    """Offsets past M or below 0 are clamped, decreasing ones leave rows
    unspecified: nothing outside the output is written, and a group whose own
    offsets are in order gets its rows."""
    import torch
    import fp8_quantized_linear_mxq_amd as mxq
    gu.say(f"grouped {pair} offsets out of range")
    rng = np.random.default_rng(4)
    n, k = 40, 128
    for m in (20, 300):
        (a, av), (w, wv) = _acts(rng, pair, m, k), _weights(rng, pair, 4 * n, k)
        guard = torch.full((m + 64, n), -7.0, dtype=torch.bfloat16, device="cuda")
        off = torch.tensor([-50, 6, 10, 10, m + 10000], dtype=torch.int32, device="cuda")
        y = mxq.gemm_grouped(a, w, off, out=guard[32:32 + m])
        g = guard.float().cpu().numpy()
        assert np.all(g[:32] == -7.0) and np.all(g[32 + m:] == -7.0)
        for e, (r0, r1) in enumerate([(0, 6), (6, 10), (10, 10), (10, m)]):
            if r1 > r0:
                gu.check_gemm(y, av[r0:r1], wv[e * n:(e + 1) * n], 1.0, rows=np.arange(r0, r1), tag="clamped")
        off = torch.tensor([15, 3, 2 ** 31 - 1, -2 ** 31, 7], dtype=torch.int32, device="cuda")
        mxq.gemm_grouped(a, w, off, out=guard[32:32 + m])
        g = guard.float().cpu().numpy()
        assert np.all(g[:32] == -7.0) and np.all(g[32 + m:] == -7.0)


def test_grouped_one_group_is_the_plain_product():
    import torch
    import fp8_quantized_linear_mxq_amd as mxq
    gu.say("grouped with one group against gemm")
    rng = np.random.default_rng(12)
    for m in (3, 200):
        (a, _), (w, _) = _acts(rng, "INT8", m, 192), _weights(rng, "INT8", 104, 192)
        off = torch.tensor([0, m], dtype=torch.int32, device="cuda")
        assert torch.equal(mxq.gemm_grouped(a, w, off), mxq.gemm(a, w))


def test_grouped_in_a_graph_with_new_offsets():
    """One captured call serves any routing: the offsets are read on replay."""
    import torch
    import fp8_quantized_linear_mxq_amd as mxq
    gu.say("grouped in a graph")
    rng = np.random.default_rng(7)
    for pair in PAIRS:
        for m in (12, 400):
            (a, _), (w, _) = _acts(rng, pair, m, 256), _weights(rng, pair, 6 * 72, 256)
            off = torch.from_numpy(_offsets([m, 0, 0, 0, 0, 0])).cuda()
            out = torch.zeros((m, 72), dtype=torch.bfloat16, device="cuda")
            mxq.gemm_grouped(a, w, off, out=out)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                mxq.gemm_grouped(a, w, off, out=out)
            for i in range(4):
                cut = np.sort(rng.integers(0, m + 1, 5))
                off.copy_(torch.from_numpy(np.concatenate([[0], cut, [m]]).astype(np.int32)))
                g.replay()
                torch.cuda.synchronize()
                assert torch.equal(out, mxq.gemm_grouped(a, w, off))


# Each tile shape that the number of tiles selects: (sizes, n, k) from a few
# 16-row tiles to two rounds of 256 x 192 and of 256 x 256
TILED = [([70, 0, 30], 100, 160), ([300, 2, 0, 350], 500, 416), ([700, 690, 0, 710], 1000, 288),
         ([1100, 1000, 0, 900], 1200, 256), ([2100, 30, 1900], 1800, 128), ([7000, 1, 6900], 2000, 128),
         ([7000, 1, 6900], 3000, 128)]


@pytest.mark.parametrize("case", range(len(TILED)))
@pytest.mark.parametrize("pair", PAIRS)
def test_grouped_tile_shapes(pair, case):
    """Against float64 products on the device."""
    import torch
    import fp8_quantized_linear_mxq_amd as mxq
    sizes, n, k = TILED[case]
    if pair != "INT8":
        k = (k + 127) // 128 * 128
    rng = np.random.default_rng(900 + case)
    off = _offsets(sizes)
    gu.say(f"grouped {pair} sizes {sizes} N={n} K={k}")
    (a, av), (w, wv) = _acts(rng, pair, int(off[-1]), k), _weights(rng, pair, len(sizes) * n, k)
    y = mxq.gemm_grouped(a, w, torch.from_numpy(off).cuda())
    for g in range(len(sizes)):
        rows = slice(int(off[g]), int(off[g + 1]))
        ad = torch.from_numpy(av[rows]).cuda()
        wd = torch.from_numpy(wv[g * n:(g + 1) * n]).cuda().t().contiguous()
        want = ad @ wd
        tol = 1e-5 * (1 + 2 ** -8) * (ad.abs() @ wd.abs()) + 2.0 ** -8 * want.abs() + 2.0 ** -133
        err = (y[rows].double() - want).abs()
        assert bool((err <= tol).all()), f"group {g}: worst {float((err / tol).max()):.3g}"
