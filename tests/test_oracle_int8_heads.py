"""Pins of the int8 and head-norm oracles: exact rationals, closed forms."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import heads, int8


def _rne(fr: Fraction) -> int:
    lo = fr.numerator // fr.denominator
    rem = fr - lo
    if rem > Fraction(1, 2) or (rem == Fraction(1, 2) and lo % 2):
        lo += 1
    return lo


@pytest.mark.parametrize("seed", range(4))
def test_int8_codes_match_exact_rationals(seed):
    rng = np.random.default_rng(seed)
    x = (rng.standard_t(3, size=(6, 64)) * 10.0 ** rng.uniform(-6, 6)).astype(np.float32)
    q, s = int8.quantize(x)
    for r in range(6):
        amax = max(abs(Fraction(float(v))) for v in x[r])
        # the float32 nearest amax / 127
        exact = amax / 127
        near = [np.nextafter(s[r], np.float32(0)), s[r], np.nextafter(s[r], np.float32(np.inf))]
        assert min(near, key=lambda c: abs(Fraction(float(c)) - exact)) == s[r]
        for k in range(64):
            assert _rne(Fraction(float(x[r, k])) / Fraction(float(s[r]))) == q[r, k]


def test_int8_closed_forms():
    # s = 1: integers are their own codes, half-integers go to even
    x = np.zeros((1, 64), np.float32)
    x[0, :8] = [127, -127, 0.5, 1.5, 2.5, -0.5, -1.5, 63.25]
    q, s = int8.quantize(x)
    assert s[0] == 1 and list(q[0, :8]) == [127, -127, 0, 2, 2, 0, -2, 63]
    q, s = int8.quantize(np.zeros((3, 32), np.float32))
    assert not q.any() and not s.any()
    # a subnormal scale still gives codes in range
    q, s = int8.quantize(np.full((1, 32), 1e-44, np.float32))
    assert np.abs(q.astype(int)).max() <= 127
    # all of a row's quotients stay within half a step
    rng = np.random.default_rng(0)
    x = rng.standard_normal((9, 96)).astype(np.float32)
    q, s = int8.quantize(x)
    assert np.all(np.abs(int8.dequantize(q, s) - x) <= s[:, None] * (0.5 + 1e-5))


@pytest.mark.parametrize("interleaved", [False, True])
def test_heads_closed_forms(interleaved):
    rng = np.random.default_rng(1)
    v = rng.standard_normal((5, 3, 16))
    # unit norm: mean square 1, and a rotation keeps every pair's length
    ang = rng.uniform(-3, 3, (5, 4))
    n = heads.norm_rope(v, eps=0.0)
    assert np.allclose((n * n).mean(axis=2), 1)
    r = heads.norm_rope(v, cos=np.cos(ang), sin=np.sin(ang), eps=0.0, interleaved=interleaved)
    assert np.allclose((r * r).sum(axis=2), (n * n).sum(axis=2))
    assert np.array_equal(r[:, :, 8:], n[:, :, 8:])      # past the rotated part
    # a quarter turn sends (a, b) to (-b, a)
    q = heads.norm_rope(v, cos=np.zeros((5, 4)), sin=np.ones((5, 4)), eps=0.0, interleaved=interleaved)
    a, b = (slice(0, 8, 2), slice(1, 8, 2)) if interleaved else (slice(0, 4), slice(4, 8))
    assert np.array_equal(q[:, :, a], -n[:, :, b]) and np.array_equal(q[:, :, b], n[:, :, a])
    # scores depend on the distance of positions only
    w = np.array([1.0, 0.3, 0.1, 0.02])
    tab = np.arange(40)[:, None] * w
    k = dict(cos=np.cos(tab), sin=np.sin(tab), eps=0.0, interleaved=interleaved)
    def score(i, j):
        x = heads.norm_rope(v[:1, :1], positions=[i], **k)
        y = heads.norm_rope(v[1:2, :1], positions=[j], **k)
        return float((x * y).sum())
    assert np.isclose(score(3, 11), score(20, 28))
