"""Pins of the FP8, gated feed-forward and layer-norm oracles: exact
rationals, closed forms, and gradients against differences."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import feed_forward as ff
from oracle import fp8
from tests import exact


@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("seed", range(3))
def test_fp8_codes_match_exact_rationals(seed, tile):
    rng = np.random.default_rng(seed)
    x = (rng.standard_t(3, size=(3, 160)) * 10.0 ** rng.uniform(-6, 6)).astype(np.float32)
    if seed == 2:   # short mantissas tie often
        x = (np.round(rng.uniform(-56, 56, x.shape)) * 2.0 ** -4).astype(np.float32)
    codes, s = fp8.quantize(x, tile)
    assert s.shape == ((1, 2) if tile else (2, 3))
    grid = exact.e4m3_grid()
    for r in range(3):
        for k in range(160):
            block = x[:, k // 128 * 128:k // 128 * 128 + 128]
            amax = np.abs(block if tile else block[r]).max()
            scale = s[0, k // 128] if tile else s[k // 128, r]
            assert Fraction(float(scale)) == exact.rn_f32(Fraction(float(amax)) / 448)
            want = exact.round_to_grid(Fraction(float(x[r, k])) / Fraction(float(scale)), grid)
            assert codes[r, k] & 0x7F == want and bool(codes[r, k] >> 7) == exact.signbit(x[r, k])


def test_fp8_closed_forms():
    x = np.zeros((2, 128), np.float32)
    x[0, :6] = [448, -448, 17, 19, 2.0 ** -9, 1.5 * 2.0 ** -9]   # scale 1: ties to even, subnormals
    codes, s = fp8.quantize(x)
    assert s[0, 0] == 1 and s[0, 1] == 0 and not codes[1].any()
    assert list(fp8.dequantize(codes, s)[0, :6]) == [448, -448, 16, 20, 2.0 ** -9, 2.0 ** -8]
    p = fp8.largest_products(np.array([[1.0] * 128 + [3.0]]), np.array([[2.0] * 128 + [-5.0]]))
    assert p[0, 0] == 2 + 15


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gated_gradients_match_differences(act):
    rng = np.random.default_rng(3)
    x, wg, wu, dy = (rng.standard_normal(s) for s in ((4, 6), (5, 6), (5, 6), (4, 5)))
    dx, dwg, dwu, _, _ = ff.gated_backward(dy, x, wg, wu, act)
    for arr, grad in ((x, dx), (wg, dwg), (wu, dwu)):
        for i in np.ndindex(arr.shape):
            keep, h = arr[i], 1e-5
            arr[i] = keep + h
            up = (ff.gated(x, wg, wu, act)[0] * dy).sum()
            arr[i] = keep - h
            down = (ff.gated(x, wg, wu, act)[0] * dy).sum()
            arr[i] = keep
            # central differences: h**2 of the third derivative, 1e-16 / h of rounding
            assert abs((up - down) / (2 * h) - grad[i]) < 1e-7


def test_activation_values():
    assert ff.activation(0.0, "silu") == 0 and np.isclose(ff.activation(1.0, "silu"), 0.7310585786300049)
    assert np.isclose(ff.activation(1.0, "gelu"), 0.8413447460685429)
    assert abs(ff.activation(1.0, "gelu_tanh") - ff.activation(1.0, "gelu")) < 5e-4
    for act in ("silu", "gelu", "gelu_tanh"):
        assert np.isclose(ff.activation(40.0, act), 40) and abs(ff.activation(-40.0, act)) < 1e-12


def test_layer_norm_closed_forms_and_differences():
    rng = np.random.default_rng(4)
    x, dy = rng.standard_normal((3, 7)) + 5, rng.standard_normal((3, 7))
    w, b = rng.standard_normal(7), rng.standard_normal(7)
    y, mean, rstd = ff.layer_norm(x, eps=0.0)
    assert np.allclose(y.mean(axis=1), 0) and np.allclose((y * y).mean(axis=1), 1)
    assert np.allclose(ff.layer_norm(3 * x + 2, eps=0.0)[0], y)
    dx, dw, db = ff.layer_norm_backward(dy, x, w)
    for arr, grad in ((x, dx), (w, dw), (b, db)):
        for i in np.ndindex(arr.shape):
            keep, h = arr[i], 1e-5
            arr[i] = keep + h
            up = (ff.layer_norm(x, w, b)[0] * dy).sum()
            arr[i] = keep - h
            down = (ff.layer_norm(x, w, b)[0] * dy).sum()
            arr[i] = keep
            assert abs((up - down) / (2 * h) - grad[i]) < 1e-7
    assert np.allclose(ff.layer_norm(np.full((1, 5), 3.0), w[:5], b[:5])[0], b[:5])
