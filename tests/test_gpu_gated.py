"""GPU parity of the gated projections and their gradients.

Exactly, where every sum is exact: the gate's pre-activations are whole numbers
of 64 and more, at which silu(g) is g and its slope 1 in fp32 to the last bit, so
the outputs and all gradients are whole numbers below 2**24, rounded once.  And
within derived bounds on random data, for every activation."""
import numpy as np
import pytest
import torch

import fp8_quantized_linear_mxq_amd as mxq
from oracle import feed_forward as ff
from oracle import fp8 as o8
from tests import gpu_util as gu
from tests.test_gpu_fp8 import bf16, gen, whole

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def sparse(g, rows, k, first, nonzeros=30):
    """Rows of -1, 0, 1 with about `nonzeros` others and `first` in column 0."""
    v = torch.randint(0, 2, (rows, k), generator=g, device="cuda").float() * 2 - 1
    v = v * (torch.rand((rows, k), generator=g, device="cuda") < min(1.0, nonzeros / k))
    v[:, 0] = first
    return v


def exact_case(m, n, k):
    """x, wg, wu, dy with g in [64, 255] and |u| < 64 (checked)."""
    g = gen(m + 3 * n + 7 * k)
    x, wg, wu = sparse(g, m, k, 1), sparse(g, n, k, 128), sparse(g, n, k, 0)
    dy = torch.randint(-1, 2, (m, n), generator=g, device="cuda").float()
    gate, up = x.double() @ wg.double().t(), x.double() @ wu.double().t()
    if m and n:
        assert 64 <= float(gate.min()) and float(gate.max()) < 256 and float(up.abs().max()) < 64
    return x, wg, wu, dy, gate, up


# single rows, odd sizes around the tiles, K that ends inside a K-tile, several tiles
SHAPES = [(1, 1, 8), (1, 200, 64), (3, 65, 72), (16, 64, 128), (17, 129, 136), (64, 64, 64), (65, 31, 200), (128, 128, 256),
          (130, 257, 1160), (300, 100, 520), (1111, 203, 160), (200, 2003, 96), (4, 3000, 1024), (2300, 1030, 264),
          (1, 513, 8192)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_forward_and_gradients_of_exact_sums(m, n, k):
    gu.say(f"gated {m}x{n}x{k} bf16, exact sums")
    x, wg, wu, dy, gate, up = exact_case(m, n, k)
    ops = [mxq.bf16_operand(t.bfloat16()) for t in (x, wg, wu)]
    saved = torch.empty((2, m, n), device="cuda")
    want = bf16(gate * up)
    assert torch.equal(mxq.gemm_gated(*ops), want)
    assert torch.equal(mxq.gemm_gated(*ops, saved=saved), want)
    assert torch.equal(saved.double(), torch.stack([gate, up]))
    dx, dwg, dwu = mxq.gemm_gated_backward(dy.bfloat16(), *ops, saved)
    dg, du = dy.double() * up, dy.double() * gate
    assert torch.equal(dx, bf16(dg @ wg.double() + du @ wu.double()))
    assert torch.equal(dwg, bf16(dg.t() @ x.double()))
    assert torch.equal(dwu, bf16(du.t() @ x.double()))


@pytest.mark.parametrize("m,n,k", [(1, 40, 32), (3, 300, 160), (20, 129, 288), (130, 257, 1184), (700, 1000, 416),
                                   (2200, 2100, 256), (5, 700, 4096)])
def test_fp8_forward_of_exact_sums(m, n, k):
    gu.say(f"gated {m}x{n}x{k} fp8, exact sums")
    g = gen(m + n + k)
    d = min(1.0, 100 / k)
    (a, av), (wg, gv), (wu, uv) = whole(g, m, k, False, -1, 2, d), whole(g, n, k, True, -1, 2, d), whole(g, n, k, True, -1, 2, d)
    for q, v, first in ((a, av, 32.0), (wg, gv, 64.0), (wu, uv, 0.0)):   # g >= 512 - what the others take off
        q.codes.view(torch.float8_e4m3fn)[:, 0] = torch.tensor(first, device="cuda").to(torch.float8_e4m3fn)
        s = (q.scales[0] if q is a else q.scales[:, 0].repeat_interleave(128)[:n]).double()
        v[:, 0] = first * s
    gate, up = av @ gv.t(), av @ uv.t()
    assert float(gate.min()) >= 64 and float((gate * up).abs().max()) < 2 ** 24 / 16   # multiples of 1/16
    assert torch.equal(mxq.gemm_gated(a, wg, wu), bf16(gate * up))


def test_parts_of_wider_tensors():
    """Operands, outputs and gradients with row strides; both projections parts
    of one matrix; what lies between is left as it was."""
    m, n, k = 70, 90, 136
    x, wg, wu, dy, gate, up = exact_case(m, n, k)
    both = torch.zeros((2 * n, k + 24), dtype=BF, device="cuda")
    both[:n, :k], both[n:, 8:8 + k] = wg.bfloat16(), wu.bfloat16()
    xs = torch.zeros((m, k + 40), dtype=BF, device="cuda")
    xs[:, 16:16 + k] = x.bfloat16()
    ops = [mxq.bf16_operand(t) for t in (xs[:, 16:16 + k], both[:n, :k], both[n:, 8:8 + k])]
    for pad in (0, 1, 2, 6):
        out = torch.full((m, n + pad), -7.0, dtype=BF, device="cuda")
        saved = torch.empty((2, m, n), device="cuda")
        mxq.gemm_gated(*ops, saved=saved, out=out)
        assert torch.equal(out[:, :n], bf16(gate * up)) and bool((out[:, n:] == -7).all())
        dys = torch.full((m, n + pad + 3), float("nan"), dtype=BF, device="cuda")
        dys[:, pad:pad + n] = dy.bfloat16()
        dx = torch.full((m, k + pad), -7.0, dtype=BF, device="cuda")
        dw = torch.full((2 * n, k + pad), -7.0, dtype=BF, device="cuda")
        got = mxq.gemm_gated_backward(dys[:, pad:pad + n], *ops, saved, dx=dx, dw_gate=dw[:n], dw_up=dw[n:])
        dg, du = dy.double() * up, dy.double() * gate
        assert got[0] is dx
        assert torch.equal(dx[:, :k], bf16(dg @ wg.double() + du @ wu.double()))
        assert torch.equal(dw[:, :k], bf16(torch.cat([dg, du], 1).t() @ x.double()))
        assert bool((dx[:, k:] == -7).all()) and bool((dw[:, k:] == -7).all())


def test_wanted_gradients_and_no_terms():
    x, wg, wu, dy, gate, up = exact_case(40, 50, 64)
    ops = [mxq.bf16_operand(t.bfloat16()) for t in (x, wg, wu)]
    saved = torch.stack([gate, up]).float()
    full = mxq.gemm_gated_backward(dy.bfloat16(), *ops, saved)
    only = mxq.gemm_gated_backward(dy.bfloat16(), *ops, saved, want=(True, False))
    assert torch.equal(only[0], full[0]) and only[1:] == (None, None)
    only = mxq.gemm_gated_backward(dy.bfloat16(), *ops, saved, want=(False, True))
    assert only[0] is None and torch.equal(only[1], full[1]) and torch.equal(only[2], full[2])
    # no rows: nothing out, zero gradients of the weights
    none = mxq.bf16_operand(torch.empty((0, 64), dtype=BF, device="cuda"))
    s0 = torch.empty((2, 0, 50), device="cuda")
    assert mxq.gemm_gated(none, *ops[1:], saved=s0).shape == (0, 50)
    dx, dwg, dwu = mxq.gemm_gated_backward(torch.empty((0, 50), dtype=BF, device="cuda"), none, *ops[1:], s0)
    assert dx.shape == (0, 64) and not dwg.any() and not dwu.any() and dwg.shape == (50, 64)
    # no outputs: a zero gradient of x
    w0 = mxq.bf16_operand(torch.empty((0, 64), dtype=BF, device="cuda"))
    dx, dwg, _ = mxq.gemm_gated_backward(torch.empty((40, 0), dtype=BF, device="cuda"), ops[0], w0, w0,
                                         torch.empty((2, 40, 0), device="cuda"))
    assert dx.shape == (40, 64) and not dx.any() and dwg.shape == (0, 64)


def _np(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("m,n,k,spread", [(1, 70, 128, 1.0), (50, 130, 200, 4.0), (33, 40, 1024, 0.3), (140, 64, 64, 12.0)])
def test_random(m, n, k, spread, act):
    """Bounds: a pre-activation's sum is off by at most 1e-5 of its absolute terms
    (fp32, K / 16 roundings of 2**-24), the activation's slope is below 1.13 and
    its own slope below 1.2, its evaluation off by at most 1e-5 |g|; dg and du are
    rounded to bf16 (2**-8 of each), outputs once more."""
    gu.say(f"gated {m}x{n}x{k} {act} spread {spread}")
    g = gen(m + n + k)
    x = torch.randn((m, k), generator=g, device="cuda").bfloat16()
    wg, wu = ((torch.randn((n, k), generator=g, device="cuda") * spread * k ** -0.5).bfloat16() for _ in range(2))
    dy = torch.randn((m, n), generator=g, device="cuda").bfloat16()
    ops = [mxq.bf16_operand(t) for t in (x, wg, wu)]
    saved = torch.empty((2, m, n), device="cuda")
    y = mxq.gemm_gated(*ops, act=act, saved=saved)
    grads = mxq.gemm_gated_backward(dy, *ops, saved, act=act)
    xn, gn, un, dn = (_np(t) for t in (x, wg, wu, dy))
    ref, gate, up = ff.gated(xn, gn, un, act)
    eg, eu = 1e-5 * (np.abs(xn) @ np.abs(gn).T), 1e-5 * (np.abs(xn) @ np.abs(un).T)
    assert np.all(np.abs(_np(saved[0]) - gate) <= eg) and np.all(np.abs(_np(saved[1]) - up) <= eu)
    ef = 1.13 * eg + 1e-5 * np.abs(gate)
    f, slope = ff.activation(gate, act), ff.activation_slope(gate, act)
    tol = ef * np.abs(up) + (np.abs(f) + ef) * eu + 2.0 ** -8 * np.abs(ref) + 2.0 ** -133
    assert np.all(np.abs(_np(y) - ref) <= tol)
    dx, dwg, dwu, dg, du = ff.gated_backward(dn, xn, gn, un, act)
    es = 1.2 * eg + 1e-5 * (1 + np.abs(gate))
    tg = np.abs(dn) * (np.abs(up) * es + (np.abs(slope) + es) * eu) + 2.0 ** -8 * np.abs(dg)
    tu = np.abs(dn) * ef + 2.0 ** -8 * np.abs(du)
    for got, want, t in ((grads[0], dx, tg @ np.abs(gn) + tu @ np.abs(un)), (grads[1], dwg, tg.T @ np.abs(xn)),
                         (grads[2], dwu, tu.T @ np.abs(xn))):
        terms = {id(dx): np.abs(dg) @ np.abs(gn) + np.abs(du) @ np.abs(un), id(dwg): np.abs(dg).T @ np.abs(xn),
                 id(dwu): np.abs(du).T @ np.abs(xn)}[id(want)]
        err = np.abs(_np(got) - want)
        assert np.all(err <= 1.01 * t + 1e-5 * terms + 2.0 ** -8 * np.abs(want) + 2.0 ** -133)
        # both roundings are half a step of 2**-7 at most and independent: in the
        # 2-norm they stay below one worst rounding
        assert np.linalg.norm(err) <= 2.0 ** -8 * np.linalg.norm(want)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_extreme_pre_activations(act):
    """Gates from -1e30 to 1e30: outputs and gradients stay finite and right."""
    gate = torch.tensor([0.0, 1e-30, 0.5, -0.5, 6, -6, 20, -20, 90, -90, 200, -200, 1e5, -1e5, 1e15, -1e15, 1e30, -1e30], device="cuda")
    gate = gate.bfloat16()
    n = len(gate)
    x = torch.zeros((2, 8), device="cuda")
    x[:, 0], x[1, 1] = 1, 1
    wg, wu = torch.zeros((n, 8), device="cuda"), torch.zeros((n, 8), device="cuda")
    wg[:, 0], wu[:, 0], wu[:, 1] = gate.float(), 1, 2
    ops = [mxq.bf16_operand(t.bfloat16()) for t in (x, wg, wu)]
    saved = torch.empty((2, 2, n), device="cuda")
    y = mxq.gemm_gated(*ops, act=act, saved=saved)
    dy = torch.ones((2, n), dtype=BF, device="cuda")
    _, dwg, dwu = mxq.gemm_gated_backward(dy, *ops, saved, act=act)
    with np.errstate(over="ignore"):
        gn = _np(gate)
        f, slope = ff.activation(gn, act), ff.activation_slope(np.clip(gn, -1e4, 1e4), act)
    close = lambda a, b, r: np.all(np.abs(a - b) <= r * np.abs(b) + 1e-6)   # noqa: E731
    assert close(_np(y[0]), f, 2.0 ** -8 + 1e-5) and close(_np(y[1]), 3 * f, 2.0 ** -8 + 1e-5)
    assert close(_np(dwg[:, 1]), 3 * slope, 2.0 ** -7 + 1e-5) and close(_np(dwu[:, 1]), f, 2.0 ** -7 + 1e-5)
    assert bool(torch.isfinite(dwg).all()) and bool(torch.isfinite(dwu).all())


def test_fp8_random():
    """The FP8 pair on quantized data, against the bound of its sums."""
    rng = np.random.default_rng(7)
    m, n, k = 40, 150, 416
    x = (rng.standard_t(3, size=(m, k)) * np.exp(rng.uniform(-2, 2, k))).astype(np.float32)
    ws = [rng.normal(0, 0.05, (n, k)).astype(np.float32) for _ in range(2)]
    qx, qw = o8.quantize(x), [o8.quantize(w, True) for w in ws]
    dev = lambda q, t: mxq.fp8_operand(torch.from_numpy(q[0]).cuda(), torch.from_numpy(q[1]).cuda(), tile=t)   # noqa: E731
    a, gv, uv = o8.dequantize(*qx), o8.dequantize(*qw[0], True), o8.dequantize(*qw[1], True)
    for act in ("silu", "gelu", "gelu_tanh"):
        y = mxq.gemm_gated(dev(qx, False), dev(qw[0], True), dev(qw[1], True), act=act)
        ref, gate, up = ff.gated(a, gv, uv, act)
        e = [2.0 ** -10 * o8.largest_products(a, w) + 1e-5 * (np.abs(a) @ np.abs(w).T) for w in (gv, uv)]
        f, ef = ff.activation(gate, act), 1.13 * e[0] + 1e-5 * np.abs(gate)
        tol = ef * np.abs(up) + (np.abs(f) + ef) * e[1] + 2.0 ** -8 * np.abs(ref) + 2.0 ** -133
        assert np.all(np.abs(_np(y) - ref) <= tol)
