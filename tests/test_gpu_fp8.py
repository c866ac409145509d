"""GPU parity of the FP8 quantizes and products: codes and scales bit for bit
against the float64 oracle; products exactly where every sum is exact (small
whole codes, power-of-two scales), and within the stated bound on random data."""
import numpy as np
import pytest
import torch

import fp8_quantized_linear_mxq_amd as mxq
from fp8_quantized_linear_mxq_amd import workloads as wl
from oracle import fp8 as o8
from oracle import hadamard as oh
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


def _check_codes(got, vals, tile, tag):
    codes, s = o8.quantize(vals, tile)
    assert np.array_equal(got.scales.cpu().numpy(), s), f"{tag}: scales"
    have = got.codes.cpu().numpy()[:, :vals.shape[1]]
    assert np.array_equal(have, codes), f"{tag}: {np.sum(have != codes)} codes differ"


# one row, rows around the 32 and the tiles of 128, columns that end inside a block
QSHAPES = [(1, 32), (3, 1152), (37, 1184), (31, 128), (33, 160), (130, 96), (128, 512), (257, 640), (5, 4128), (1030, 544)]


@pytest.mark.parametrize("rows,cols", QSHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["FP8", "FP8_TILE"])
def test_quantize(rows, cols, dtype, fmt):
    gu.say(f"{fmt} quantize {rows}x{cols} {dtype}")
    rng = np.random.default_rng(rows + cols)
    x = (rng.standard_t(3, size=(rows, cols)) * np.exp(rng.uniform(-5, 5, size=cols))).astype(np.float32)
    x = wl.f32_to_bf16_bits(x) if dtype == "bf16" else x
    got = mxq.quantize(gu.act_to_dev(x, dtype), mxq.FORMATS[fmt])
    _check_codes(got, gu.act_values(x, dtype), fmt == "FP8_TILE", f"{rows}x{cols}")


@pytest.mark.parametrize("had", [16, 32, 128])
@pytest.mark.parametrize("fmt", ["FP8", "FP8_TILE"])
def test_quantize_rotated(had, fmt):
    gu.say(f"{fmt} quantize rotated by {had}")
    rng = np.random.default_rng(had)
    bits = wl.f32_to_bf16_bits(rng.standard_t(4, size=(140, 384 if had == 128 else 416)).astype(np.float32))
    want = oh.rotate(wl.bf16_to_f32(bits), had, 7)
    for dev in (gu.to_dev_bf16(bits), gu.to_dev_f32(wl.bf16_to_f32(bits))):
        _check_codes(mxq.quantize(dev, mxq.FORMATS[fmt], hadamard=had), want, fmt == "FP8_TILE", f"rotated {had}")


@pytest.mark.parametrize("fmt", ["FP8", "FP8_TILE"])
def test_quantize_ties_zeros_and_small_blocks(fmt):
    """Middles between codes and their neighbours under exact and odd scales,
    subnormal codes, zero blocks, scales that are subnormal or underflow."""
    rng = np.random.default_rng(9)
    grid = np.array([o for o in o8.E4M3.decode(np.arange(127))])
    mid = np.concatenate([(grid[1:] + grid[:-1]) / 2, grid])[:252]
    rows = []
    for r in range(24):
        s = 2.0 ** (3 * r - 20) if r < 8 else rng.uniform(0.5, 2) * 2.0 ** (-12 * (r - 8))
        v = np.zeros(256)
        v[:252] = mid * s * np.where(rng.random(252) < 0.5, -1, 1)
        v = v.astype(np.float32)
        if r % 3 == 1:
            v = np.nextafter(v, np.float32(np.inf))
        if r % 3 == 2:
            v = np.nextafter(v, np.float32(-np.inf))
        v[[126, 252]] = np.float32(448 * s)
        rows.append(v)
    rows += [np.zeros(256), np.full(256, 1e-44), np.full(256, -1.4e-45), np.full(256, 3e38), np.full(256, -0.0)]
    x = np.array(rows, np.float32)
    if fmt == "FP8_TILE":   # each row a tile of its own
        for r in x:
            _check_codes(mxq.quantize(gu.to_dev_f32(r[None]), mxq.FP8_TILE), r[None], True, "row")
    else:
        _check_codes(mxq.quantize(gu.to_dev_f32(x), mxq.FP8), x, False, "rows")


def test_quantize_strides_and_given_output():
    """Rows of a wider tensor; codes and scales in parts of larger ones, which keep their other values."""
    rng = np.random.default_rng(1)
    x = gu.to_dev_f32(rng.standard_normal((70, 400)).astype(np.float32))[:, 16:16 + 288]
    codes = torch.full((70, 320), 77, dtype=torch.uint8, device="cuda")
    scales = torch.full((4, 90), -5.0, device="cuda")
    q = mxq.QTensor(mxq.FP8, 70, 288, codes, scales[:, 7:77])
    mxq.quantize(x, mxq.FP8, out=q)
    want, s = o8.quantize(x.cpu().numpy())
    assert np.array_equal(codes[:, :288].cpu().numpy(), want) and bool((codes[:, 288:] == 77).all())
    assert np.array_equal(scales[:3, 7:77].cpu().numpy(), s)
    assert bool((scales[3] == -5).all()) and bool((scales[:, :7] == -5).all()) and bool((scales[:, 77:] == -5).all())


# ---- products -------------------------------------------------------------

def whole(g, rows, k, tile, lo=-3, hi=4, density=1.0):
    """Codes of small whole numbers and power-of-two scales: (operand, float64 values)."""
    v = torch.randint(lo, hi, (rows, k), generator=g, device="cuda").float()
    if density < 1:
        v = v * (torch.rand((rows, k), generator=g, device="cuda") < density)
    kb = (k + 127) // 128
    shape = ((rows + 127) // 128, kb) if tile else (kb, rows)
    s = torch.exp2(torch.randint(-1, 2, shape, generator=g, device="cuda").float())
    d = s.double() if tile else s.t().double()
    d = (d.repeat_interleave(128, 0)[:rows] if tile else d).repeat_interleave(128, 1)[:, :k]
    return mxq.fp8_operand(v.to(torch.float8_e4m3fn), s, tile=tile), v.double() * d


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def bf16(v):
    return v.float().bfloat16()   # v fits float32


# single rows and columns, sizes around the tiles, K inside a block, long K, many tiles
SHAPES = [(1, 1, 32), (1, 300, 128), (16, 40, 96), (17, 129, 160), (64, 64, 256), (65, 200, 416), (128, 128, 1152),
          (129, 1001, 224), (300, 257, 1184), (777, 1001, 1184), (256, 256, 4096), (1, 4096, 4096), (30, 2000, 8192),
          (2500, 2100, 640), (5000, 3, 288), (3, 5000, 288), (4100, 4096, 512)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gemm_of_exact_sums(m, n, k):
    gu.say(f"fp8 gemm {m}x{n}x{k}, exact sums")
    g = gen(m + n + k)
    (a, av), (w, wv) = whole(g, m, k, False), whole(g, n, k, True)
    assert torch.equal(mxq.gemm(a, w), bf16(av @ wv.t()))


@pytest.mark.parametrize("m,n,k", [(5, 70, 160), (150, 141, 288), (300, 520, 256)])
def test_gemm_bias_map_and_strides(m, n, k):
    gu.say(f"fp8 gemm {m}x{n}x{k}: bias, column map, strides")
    g = gen(m)
    (a, av), (w, wv) = whole(g, m, k, False), whole(g, n, k, True)
    bias = torch.randint(-9, 9, (n + 6,), generator=g, device="cuda").bfloat16()
    y = av @ wv.t()
    assert torch.equal(mxq.gemm(a, w, bias=bias[:n]), bf16(y + bias[:n].double()))
    for pad in (0, 1, 2, 5, 8):
        out = torch.full((m, n + pad), -7.0, dtype=torch.bfloat16, device="cuda")
        mxq.gemm(a, w, out=out)
        assert torch.equal(out[:, :n], bf16(y)) and bool((out[:, n:] == -7).all())
    perm = torch.randperm(n + 6, generator=g, device="cuda")[:n].int()
    perm[n // 2] = -1                                            # skipped
    out = torch.full((m, n + 6), -7.0, dtype=torch.bfloat16, device="cuda")
    mxq.gemm(a, w, n_out=n + 6, w_out_col=perm, bias=bias, out=out)
    want = torch.full((m, n + 6), -7.0, dtype=torch.bfloat16, device="cuda")
    keep = perm >= 0
    cols = perm[keep].long()
    want[:, cols] = bf16(y[:, keep] + bias[cols].double())
    assert torch.equal(out, want)
    # codes and scales inside wider tensors
    wide = torch.zeros((m, k + 64), dtype=torch.uint8, device="cuda")
    wide[:, 16:16 + k] = a.codes.view(torch.uint8)
    ws = torch.zeros((a.scales.shape[0], m + 9), device="cuda")
    ws[:, 4:4 + m] = a.scales
    a2 = mxq.fp8_operand(wide[:, 16:16 + k], ws[:, 4:4 + m])
    assert torch.equal(mxq.gemm(a2, w), bf16(y))


def test_gemm_mixed_groups():
    g = gen(2)
    (a, av), (w1, v1), (w2, v2) = whole(g, 40, 256, False), whole(g, 30, 256, True), whole(g, 50, 256, True)
    perm = torch.randperm(80, generator=g, device="cuda").int()
    want = torch.empty((40, 80), dtype=torch.bfloat16, device="cuda")
    want[:, perm.long()] = bf16(av @ torch.cat([v1, v2]).t())
    assert torch.equal(mxq.gemm_mixed(a, [w1, w2], perm, 80), want)


@pytest.mark.parametrize("m,n,k", [(1, 200, 1152), (40, 90, 1184), (200, 150, 512), (12, 64, 4096)])
def test_gemm_random(m, n, k):
    """Heavy-tailed activations against the bound of the matrix cores' sums."""
    gu.say(f"fp8 gemm {m}x{n}x{k}, random")
    rng = np.random.default_rng(m + k)
    x = (rng.standard_t(3, size=(m, k)) * np.exp(rng.uniform(-3, 3, k))).astype(np.float32)
    w = rng.normal(0, 0.02, (n, k)).astype(np.float32)
    (cx, sx), (cw, sw) = o8.quantize(x), o8.quantize(w, True)
    a, b = o8.dequantize(cx, sx), o8.dequantize(cw, sw, True)
    y = mxq.gemm(mxq.fp8_operand(torch.from_numpy(cx).cuda(), torch.from_numpy(sx).cuda()),
                 mxq.fp8_operand(torch.from_numpy(cw).cuda(), torch.from_numpy(sw).cuda(), tile=True))
    ref = a @ b.T
    err = np.abs(y.double().cpu().numpy() - ref)
    assert np.all(err <= o8.tolerance(ref, a, b)), f"worst {np.max(err / o8.tolerance(ref, a, b)):.3g} of the bound"


@pytest.mark.parametrize("sizes,n,k", [([1], 128, 128), ([0, 5, 0, 16, 17, 1], 256, 160), ([127, 128, 129, 0, 1, 300], 384, 288),
                                       ([3, 0] * 40, 128, 512), ([1000, 0, 1500, 70], 1280, 1056)])
def test_grouped(sizes, n, k):
    gu.say(f"fp8 grouped {sizes[:8]} N={n} K={k}")
    g = gen(n + k)
    first, extra = 3, 4
    off = torch.tensor([first] + [first + sum(sizes[:i + 1]) for i in range(len(sizes))], dtype=torch.int32, device="cuda")
    m, e = first + sum(sizes) + extra, len(sizes)
    (a, av), (w, wv) = whole(g, m, k, False), whole(g, e * n, k, True)
    bias = torch.randint(-9, 9, (e, n), generator=g, device="cuda").bfloat16()
    out = torch.full((m, n + 8), -7.0, dtype=torch.bfloat16, device="cuda")
    want = out.clone()
    for i in range(e):
        r = slice(int(off[i]), int(off[i + 1]))
        want[r, :n] = bf16(av[r] @ wv[i * n:(i + 1) * n].t() + bias[i].double())
    mxq.gemm_grouped(a, w, off, bias=bias, out=out)
    assert torch.equal(out, want)


def test_quantize_then_gemm_equals_its_parts():
    """The layer as a program calls it: what quantize writes is what gemm reads."""
    g = gen(5)
    x, w = torch.randn((50, 416), generator=g, device="cuda"), torch.randn((70, 416), generator=g, device="cuda")
    y = mxq.gemm(mxq.quantize(x, mxq.FP8), mxq.quantize(w, mxq.FP8_TILE))
    (cx, sx), (cw, sw) = o8.quantize(x.cpu().numpy()), o8.quantize(w.cpu().numpy(), True)
    a, b = o8.dequantize(cx, sx), o8.dequantize(cw, sw, True)
    ref = a @ b.T
    assert np.all(np.abs(y.double().cpu().numpy() - ref) <= o8.tolerance(ref, a, b))
