"""Row-wise symmetric int8 quantization in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Definition: s = RN_fp32(max |x| / 127) per row (the float64 quotient of two
float32 values rounds correctly to float32), q = clamp(RNE(x / s), -127, 127)
on the exact real quotient (the float64 quotient decides every case: x / s is
either a half-integer or at least 2**-25 away from one), s = 0 gives q = 0.
"""

from __future__ import annotations

import numpy as np


def quantize(x: np.ndarray):
    """(codes int8 [rows, K], scales float32 [rows])."""
    x = np.asarray(x, dtype=np.float32).astype(np.float64)
    amax = np.abs(x).max(axis=1) if x.shape[1] else np.zeros(x.shape[0])
    s = (amax / 127.0).astype(np.float32)
    d = np.where(s == 0, 1.0, s.astype(np.float64))[:, None]
    q = np.where(s[:, None] == 0, 0.0, np.clip(np.rint(x / d), -127, 127))
    return q.astype(np.int8), s


def dequantize(q: np.ndarray, s: np.ndarray) -> np.ndarray:
    """The exact values q * s as float64."""
    return q.astype(np.float64) * np.asarray(s, np.float64).reshape(-1, 1)
