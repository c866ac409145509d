"""GPU parity of the layer norm and its gradients against float64."""
import numpy as np
import pytest
import torch

import fp8_quantized_linear_mxq_amd as mxq
from oracle import feed_forward as ff
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _np(t):
    return t.double().cpu().numpy()


def draw(rows, cols, dtype, seed, mean=0.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")   # noqa: E731
    x = (r(rows, cols) * torch.exp(r(cols)) + mean).to(DT[dtype])
    return x, (1 + 0.2 * r(cols)).to(DT[dtype]), (0.3 * r(cols)).to(DT[dtype]), r(rows, cols).to(DT[dtype])


def steps(cols):
    """Roundings that a sum of a row passes, in units of 2**-24 of its absolute
    terms: a lane's own (at most cols / 512 + 64) and the joins of lanes and waves."""
    return (cols / 512 + 64 + 9) * 2.0 ** -24


def half(dtype):
    return 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24


def check_forward(y, x, w, b, dtype, eps=1e-5):
    xn, wn, bn = _np(x), _np(w) if w is not None else None, _np(b) if b is not None else None
    ref, mean, rstd = ff.layer_norm(xn, wn, bn, eps)
    u = steps(x.shape[1])
    h = np.abs((xn - mean) * rstd)
    # the mean's error, and that of the mean square, through h; a few roundings on the way
    eh = rstd * u * np.abs(xn).mean(axis=1, keepdims=True) * (1 + h) + h * (u + 2.0 ** -20) + rstd * np.abs(xn) * 2.0 ** -24
    tol = eh * (1 if wn is None else np.abs(wn)) + (0 if bn is None else np.abs(bn) * 2.0 ** -23)
    err = np.abs(_np(y) - ref)
    tol = tol + (half(dtype) + 2.0 ** -23) * np.abs(ref) + 2.0 ** -133
    assert np.all(err <= tol), f"worst {np.max(err / tol):.3g} of the bound"
    return mean, rstd


# every shape of the kernels: pieces of eight and single elements, one to eight waves
# to a row, rows too long for the registers; rows of one element
COLS = [1, 2, 7, 8, 63, 65, 100, 130, 257, 500, 504, 513, 1000, 1023, 1152, 2040, 2047, 2050, 4096, 4100, 4104, 8000, 8192,
        8193, 8200, 12345, 16384, 16400, 33000]


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward_and_gradients(cols, dtype):
    rows = 7 if cols > 5000 else 37
    gu.say(f"layer norm {rows}x{cols} {dtype}")
    x, w, b, dy = draw(rows, cols, dtype, cols, mean=0.5)
    stats = torch.empty((rows, 2), device="cuda")
    y = mxq.layer_norm(x, w, b, stats=stats)
    mean, rstd = check_forward(y, x, w, b, dtype)
    u = steps(cols)
    assert np.all(np.abs(_np(stats)[:, :1] - mean) <= u * np.abs(_np(x)).mean(axis=1, keepdims=True) + 1e-30)
    assert torch.equal(y, mxq.layer_norm(x, w, b))   # with and without statistics
    check_gradients(x, w, dy, stats, dtype)


def check_gradients(x, w, dy, stats, dtype, eps=1e-5):
    dx, dw, db = mxq.layer_norm_backward(dy, x, stats, w)
    rows, cols = x.shape
    xn, dn, wn = _np(x), _np(dy), _np(w) if w is not None else 1.0
    rx, rw, rb = ff.layer_norm_backward(dn, xn, None if w is None else wn, eps)
    h, mean, rstd = ff.layer_norm(xn, eps=eps)
    t, u = np.abs(dn * wn), steps(cols)
    eh = rstd * u * np.abs(xn).mean(axis=1, keepdims=True) * (1 + np.abs(h)) + np.abs(h) * (u + 2.0 ** -20) + \
        rstd * np.abs(xn) * 2.0 ** -24
    m1, m2 = t.mean(axis=1, keepdims=True), (t * np.abs(h)).mean(axis=1, keepdims=True)
    ex = rstd * ((u + 2.0 ** -20) * (t + m1 + np.abs(h) * m2) + eh * m2 + np.abs(h) * (t * eh).mean(axis=1, keepdims=True))
    tol = ex + (u + 2.0 ** -20 + half(dtype)) * np.abs(rx) + 2.0 ** -133
    err = np.abs(_np(dx) - rx)
    assert np.all(err <= tol), f"dx: worst {np.max(err / tol):.3g} of the bound"
    # sums over rows: a workgroup's own rows, then those of at most 512 workgroups by 16 waves
    v = (rows / 512 + 8 + 32 + 16) * 2.0 ** -24
    tw = (v + 2.0 ** -22) * np.abs(dn * h).sum(axis=0) + (np.abs(dn) * eh).sum(axis=0)
    assert np.all(np.abs(_np(dw) - rw) <= tw + half(dtype) * np.abs(rw) + 2.0 ** -133)
    assert np.all(np.abs(_np(db) - rb) <= v * np.abs(dn).sum(axis=0) + half(dtype) * np.abs(rb) + 2.0 ** -133)
    return dx, dw, db


@pytest.mark.parametrize("rows,cols", [(1, 4096), (2, 96), (513, 64), (1500, 520), (4100, 24), (5000, 1), (1030, 2048),
                                       (3000, 33), (700, 4097)])
def test_many_rows(rows, cols):
    """More rows than workgroups, fewer, and ends inside a workgroup's rows."""
    gu.say(f"layer norm {rows}x{cols}")
    x, w, b, dy = draw(rows, cols, "bf16", rows)
    stats = torch.empty((rows, 2), device="cuda")
    check_forward(mxq.layer_norm(x, w, b, stats=stats), x, w, b, "bf16")
    first = check_gradients(x, w, dy, stats, "bf16")
    again = mxq.layer_norm_backward(dy, x, stats, w)
    assert all(torch.equal(p, q) for p, q in zip(first, again))   # no atomics: the same bits


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_without_parameters_large_means_and_constant_rows(dtype):
    x, w, b, dy = draw(20, 640, dtype, 3)
    stats = torch.empty((20, 2), device="cuda")
    check_forward(mxq.layer_norm(x, stats=stats), x, None, None, dtype)
    check_gradients(x, None, dy, stats, dtype)
    check_forward(mxq.layer_norm(x, w), x, w, None, dtype)
    check_forward(mxq.layer_norm(x, None, b), x, None, b, dtype)
    far = (x.float() + 1000).to(DT[dtype])   # the variance is a millionth of the mean square
    check_forward(mxq.layer_norm(far, w, b), far, w, b, dtype)
    flat = torch.full((3, 640), 2.5, dtype=DT[dtype], device="cuda")
    assert torch.equal(mxq.layer_norm(flat, w, b), b.expand(3, -1))
    check_forward(mxq.layer_norm(x, w, b, eps=0.0), x, w, b, dtype, eps=0.0)
    check_forward(mxq.layer_norm(x, w, b, eps=0.3), x, w, b, dtype, eps=0.3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_alignment_and_in_place(dtype):
    x, w, b, dy = draw(33, 264, dtype, 5)
    want = mxq.layer_norm(x, w, b)
    stats = torch.empty((33, 2), device="cuda")
    mxq.layer_norm(x, w, b, stats=stats)
    grads = mxq.layer_norm_backward(dy, x, stats, w)
    for first, width in ((0, 264), (8, 280), (1, 265), (3, 271)):
        wide = torch.full((33, width + 8), float("nan"), dtype=DT[dtype], device="cuda")
        wide[:, first:first + 264] = x
        out = torch.full((33, width + 8), -7.0, dtype=DT[dtype], device="cuda")
        mxq.layer_norm(wide[:, first:first + 264], w, b, out=out[:, first:first + 264])
        tol = 1e-6 if dtype == "f32" else 2.0 ** -7
        assert torch.allclose(out[:, first:first + 264].float(), want.float(), rtol=tol, atol=1e-5)
        assert bool((out[:, :first] == -7).all()) and bool((out[:, first + 264:] == -7).all())
        wdy = torch.full_like(wide, float("nan"))
        wdy[:, first:first + 264] = dy
        wdx = torch.full_like(out, -7.0)
        got = mxq.layer_norm_backward(wdy[:, first:first + 264], wide[:, first:first + 264], stats, w,
                                      dx=wdx[:, first:first + 264])
        for p, q in zip(got, grads):
            assert torch.allclose(p.float(), q.float(), rtol=2 * tol, atol=2e-5 if dtype == "f32" else 2e-2)
        assert bool((wdx[:, :first] == -7).all()) and bool((wdx[:, first + 264:] == -7).all())
    y = x.clone()
    assert mxq.layer_norm(y, w, b, out=y) is y and torch.equal(y, want)
    for into in ("dy", "x"):
        xx, dd = x.clone(), dy.clone()
        got = mxq.layer_norm_backward(dd, xx, stats, w, dx=dd if into == "dy" else xx)
        assert all(torch.equal(p, q) for p, q in zip(got, grads))


def test_wanted_gradients_and_no_rows():
    x, w, b, dy = draw(30, 136, "bf16", 8)
    stats = torch.empty((30, 2), device="cuda")
    mxq.layer_norm(x, w, b, stats=stats)
    full = mxq.layer_norm_backward(dy, x, stats, w)
    only = mxq.layer_norm_backward(dy, x, stats, w, want=(True, False))
    assert torch.equal(only[0], full[0]) and only[1:] == (None, None)
    only = mxq.layer_norm_backward(dy, x, stats, w, want=(False, True))
    assert only[0] is None and torch.equal(only[1], full[1]) and torch.equal(only[2], full[2])
    none = x[:0]
    assert mxq.layer_norm(none, w, b).shape == (0, 136)
    dx, dw, db = mxq.layer_norm_backward(none, none, stats[:0], w)
    assert dx.shape == (0, 136) and not dw.any() and not db.any()
