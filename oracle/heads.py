"""Per-head RMS norm with the position rotation, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

n = v / sqrt(mean(v^2) + eps) * g; each pair (a, b) of the first R elements of
n becomes (a cos - b sin, b cos + a sin) -- pairs (i, i + R/2), or (2i, 2i + 1)
when interleaved -- with cos, sin row `position` of the tables; the elements
past R stay as they are.
"""

from __future__ import annotations

import numpy as np


def norm_rope(v, gain=None, cos=None, sin=None, positions=None, eps=1e-6, interleaved=False):
    """v [tokens, heads, D] -> the same shape, float64."""
    v = np.asarray(v, np.float64)
    n = v / np.sqrt(np.mean(v * v, axis=2, keepdims=True) + eps)
    if gain is not None:
        n = n * np.asarray(gain, np.float64)
    if cos is None:
        return n
    half = cos.shape[1]
    pos = np.arange(v.shape[0]) if positions is None else np.asarray(positions)
    out = n.copy()
    for t in range(v.shape[0]):
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            c, s = float(cos[pos[t], i]), float(sin[pos[t], i])
            out[t, :, a] = n[t, :, a] * c - n[t, :, b] * s
            out[t, :, b] = n[t, :, b] * c + n[t, :, a] * s
    return out
