"""NaN and infinities in the FP8 layer, the gated products, their gradients and the layer
norm: what the formulas give, and nothing in rows and columns beside them."""
import pytest
import torch

import fp8_quantized_linear_mxq_amd as mxq
from tests import gpu_util as gu
from tests.test_gpu_fp8 import bf16, gen, whole
from tests.test_gpu_gated import exact_case

pytestmark = pytest.mark.gpu

ACTS = ["silu", "gelu", "gelu_tanh"]
NAN, INF = float("nan"), float("inf")


def same(got, want):
    """Equal, NaN where the other is NaN."""
    return torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(nan=0.0), want.nan_to_num(nan=0.0))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n", [(40, 64), (40, 51)])   # eight columns and two columns to a thread
def test_nan_gate(m, n, act):
    """A NaN gate makes its outputs' gradients NaN: f'(g) is."""
    x, wg, wu, dy, gate, up = exact_case(m, n, 64)
    ops = [mxq.bf16_operand(t.bfloat16()) for t in (x, wg, wu)]
    saved = torch.stack([gate, up]).float()
    clean = mxq.gemm_gated_backward(dy.bfloat16(), *ops, saved, act=act)
    saved[0, 7, 5] = NAN
    dx, dwg, dwu = mxq.gemm_gated_backward(dy.bfloat16(), *ops, saved, act=act)
    assert bool(dx[7].isnan().all()) and bool(dwg[5].isnan().all()) and bool(dwu[5].isnan().all())
    rows, outs = torch.arange(m, device="cuda") != 7, torch.arange(n, device="cuda") != 5
    assert torch.equal(dx[rows], clean[0][rows])
    assert torch.equal(dwg[outs], clean[1][outs]) and torch.equal(dwu[outs], clean[2][outs])


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m", [3, 200])   # few rows, tiles
def test_nan_input(m, act):
    """A NaN of x reaches its row of the outputs and of the pre-activations, and no other."""
    x, wg, wu, dy, gate, up = exact_case(m, 300, 136)
    ops = [mxq.bf16_operand(t.bfloat16()) for t in (x, wg, wu)]
    clean, saved = mxq.gemm_gated(*ops, act=act), torch.empty((2, m, 300), device="cuda")
    ops[0].codes[1, 70] = NAN
    y = mxq.gemm_gated(*ops, act=act, saved=saved)
    others = torch.arange(m, device="cuda") != 1
    assert bool(y[1].isnan().all()) and bool(saved[:, 1].isnan().all())
    assert torch.equal(y[others], clean[others]) and bool(saved[:, others].isfinite().all())


def with_infinite_row(a, b, col):
    """a^T-like product a [r, t] @ b [t, c] whose last row of b is infinite in column col, the rest finite."""
    finite = b.clone()
    finite[-1, col] = 0
    want = a @ finite
    want[:, col] += a[:, -1] * b[-1, col]
    return bf16(want)


# a few rows, one and several tiles, K split over workgroups, the largest tiles; all with padded rows and outputs
@pytest.mark.parametrize("m,n,k", [(5, 9, 72), (70, 90, 136), (300, 100, 520), (1111, 203, 160), (2300, 1030, 264),
                                   (8200, 2100, 2056), (64, 128, 136)])
def test_infinite_last_rows(m, n, k):
    """Infinities in the last row of x and of the weights, behind which the operands end
    inside a K-tile: the gradients are infinite (NaN where the formula has 0 x inf)."""
    gu.say(f"gradients {m}x{n}x{k}, infinite last rows")
    x, wg, wu, dy, gate, up = exact_case(m, n, k)
    saved = torch.stack([gate, up]).float()
    dg, du = dy.double() * up, dy.double() * gate
    x[-1, 3], wg[-1, 4], wu[-1, 5] = INF, -INF, INF
    ops = [mxq.bf16_operand(t.bfloat16()) for t in (x, wg, wu)]
    dx, dwg, dwu = mxq.gemm_gated_backward(dy.bfloat16(), *ops, saved)
    xd, gd, ud = x.double(), wg.double(), wu.double()
    both = torch.cat([dg, du], 1)
    gd0, ud0 = gd.clone(), ud.clone()
    gd0[-1, 4] = ud0[-1, 5] = 0
    want = both @ torch.cat([gd0, ud0])
    want[:, 4] += dg[:, -1] * gd[-1, 4]
    want[:, 5] += du[:, -1] * ud[-1, 5]
    assert same(dx, bf16(want)), "dx"
    assert same(dwg, with_infinite_row(dg.t(), xd, 3)), "dWg"
    assert same(dwu, with_infinite_row(du.t(), xd, 3)), "dWu"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", [mxq.FP8, mxq.FP8_TILE])
def test_quantize_of_nonfinite_blocks(dtype, fmt):
    """The scale of a block with an infinity is infinite, its elements 448 (the infinite
    ones) and 0; that of a block with a NaN is NaN.  No code is NaN, and other blocks
    are as without them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    x = torch.randn((140, 416), generator=g, device="cuda").to(dtype)
    clean, y = mxq.quantize(x, fmt), x.clone()
    y[2, 140], y[129, 400], y[130, 30] = INF, -INF, NAN
    q = mxq.quantize(y, fmt)
    by_row = lambda t: t if fmt == mxq.FP8_TILE else t.t()   # noqa: E731
    scales, first = by_row(q.scales), by_row(clean.scales)
    hit = torch.zeros_like(scales, dtype=torch.bool)
    row = lambda r: r // 128 if fmt == mxq.FP8_TILE else r   # noqa: E731
    hit[row(2), 1] = hit[row(129), 3] = hit[row(130), 0] = True
    assert torch.equal(scales[~hit], first[~hit])
    assert scales[row(2), 1] == INF and scales[row(129), 3] == INF and bool(scales[row(130), 0].isnan())
    spread = (hit.repeat_interleave(128, 0)[:140] if fmt == mxq.FP8_TILE else hit).repeat_interleave(128, 1)[:, :416]
    assert torch.equal(q.codes[~spread], clean.codes[~spread])
    assert not bool(((q.codes & 127) == 127).any())
    infinite = spread & ~(scales.isnan().repeat_interleave(128, 0)[:140] if fmt == mxq.FP8_TILE
                          else scales.isnan()).repeat_interleave(128, 1)[:, :416]
    want = torch.where(y.isinf(), 126, 0).to(torch.uint8) | torch.where(torch.signbit(y), 128, 0).to(torch.uint8)
    assert torch.equal(q.codes[infinite], want[infinite])


@pytest.mark.parametrize("fmt", [mxq.FP8, mxq.FP8_TILE])
@pytest.mark.parametrize("had", [16, 128])
def test_quantize_rotates_a_nan_into_its_block(fmt, had):
    """Sums with a NaN (or of opposite infinities) are NaN: so is their block's scale, and no code is."""
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x = torch.randn((140, 384), generator=g, device="cuda")
    clean, y = mxq.quantize(x, fmt, hadamard=had), x.clone()
    y[3, 200], y[135, 1], y[135, 2] = NAN, INF, -INF
    q = mxq.quantize(y, fmt, hadamard=had)
    scales, first = (t.scales if fmt == mxq.FP8_TILE else t.scales.t() for t in (q, clean))
    hit = torch.zeros_like(scales, dtype=torch.bool)
    row = lambda r: r // 128 if fmt == mxq.FP8_TILE else r   # noqa: E731
    hit[row(3), 1] = hit[row(135), 0] = True
    assert bool(scales[hit].isnan().all()) and torch.equal(scales[~hit], first[~hit])
    assert not bool(((q.codes & 127) == 127).any())


@pytest.mark.parametrize("m,n,k", [(3, 300, 160), (200, 700, 1184), (2100, 2050, 288)])   # few rows, small and large tiles
def test_fp8_products_keep_nonfinite_scales_to_their_rows_and_tiles(m, n, k):
    """A NaN or infinite scale reaches its row of outputs, or its tile's columns, alone:
    also from the last rows, which tiles past the end read again."""
    gu.say(f"fp8 {m}x{n}x{k}, non-finite scales")
    g = gen(m + n)
    (a, av), (w, wv) = whole(g, m, k, False), whole(g, n, k, True)
    want = bf16(av @ wv.t())
    a.scales[0, m - 1], w.scales[0, 0] = NAN, INF
    y = mxq.gemm(a, w)
    assert bool(y[m - 1].isnan().all()) and not bool(y[:, :min(128, n)].isfinite().any())
    assert torch.equal(y[:m - 1, 128:], want[:m - 1, 128:])
    a.scales[0, m - 1], w.scales[0, 0], w.scales[-1, -1] = 1, 1, NAN
    y, first = mxq.gemm(a, w), (n - 1) // 128 * 128
    assert bool(y[:, first:].isnan().all()) and bool(y[:, :first].isfinite().all())


@pytest.mark.parametrize("cols", [100, 264, 1030, 2048, 16392, 16401])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_layer_norm_keeps_nonfinite_rows_to_themselves(cols, bad):
    """Also the last row, which groups of waves without a row of their own read."""
    rows = 37
    g = torch.Generator(device="cuda")
    g.manual_seed(cols)
    x, dy = (torch.randn((rows, cols), generator=g, device="cuda").bfloat16() for _ in range(2))
    stats = torch.empty((rows, 2), device="cuda")
    y = mxq.layer_norm(x, stats=stats)
    dx, dw, _ = mxq.layer_norm_backward(dy, x, stats)
    z = x.clone()
    z[5, cols // 2] = z[rows - 1, cols - 1] = bad
    other = torch.ones(rows, dtype=torch.bool, device="cuda")
    other[5] = other[rows - 1] = False
    got = mxq.layer_norm(z, stats=stats)
    assert torch.equal(got[other], y[other]) and bool(got[~other].isnan().all())
    gx, gw, _ = mxq.layer_norm_backward(dy, z, stats)
    assert torch.equal(gx[other], dx[other]) and bool(gx[~other].isnan().all()) and bool(gw.isnan().all())
    clean = torch.where(other[:, None], dy, torch.zeros_like(dy))   # a padded row's dy is zero: its NaN still is one
    assert torch.equal(mxq.layer_norm_backward(clean, z, stats)[0][other], dx[other])
