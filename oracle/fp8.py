"""E4M3 quantization with one float32 scale per block of 128 columns, of one
row or of 128 rows, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Definition: s = RN_fp32(max |x| / 448) over the block (the float64 quotient of
two float32 values rounds correctly to float32), q = RNE_E4M3(x / s) on the
exact real quotient: the float64 quotient decides every case, since x / s either
is a middle between two codes (at most 5 significant bits) or lies at least
2**-30 of itself away from one.  s = 0 gives zeros with x's sign.
"""

from __future__ import annotations

import numpy as np

from .formats import E4M3

BLOCK = 128


def spread(s: np.ndarray, rows: int, cols: int, tile: bool) -> np.ndarray:
    """The scale of every element: s [K / 128, rows], or [rows / 128, K / 128]."""
    s = np.asarray(s, np.float64)
    if tile:
        return np.repeat(np.repeat(s, BLOCK, axis=0)[:rows], BLOCK, axis=1)[:, :cols]
    return np.repeat(s.T, BLOCK, axis=1)[:, :cols]


def quantize(x: np.ndarray, tile: bool = False):
    """(codes uint8 [rows, K], scales float32 as stored)."""
    x = np.asarray(x, np.float32).astype(np.float64)
    rows, cols = x.shape
    kb, rb = -(-cols // BLOCK), -(-rows // BLOCK)
    s = np.zeros((rb, kb) if tile else (kb, rows), np.float32)
    for j in range(kb):
        top = np.abs(x[:, BLOCK * j:BLOCK * (j + 1)]).max(axis=1)
        if tile:
            for i in range(rb):
                s[i, j] = np.float32(top[BLOCK * i:BLOCK * (i + 1)].max() / 448.0)
        else:
            s[j] = (top / 448.0).astype(np.float32)
    d = spread(s, rows, cols, tile)
    q = np.where(d > 0, x / np.where(d > 0, d, 1.0), 0.0)
    return E4M3.encode(np.where(d > 0, q, np.copysign(0.0, x))), s


def dequantize(codes: np.ndarray, s: np.ndarray, tile: bool = False) -> np.ndarray:
    """The exact values code * s as float64."""
    return E4M3.decode(codes) * spread(s, *codes.shape, tile)


def largest_products(a: np.ndarray, w: np.ndarray) -> np.ndarray:
    """P [M, N]: over the K-blocks, the sum of the largest |a w| of each."""
    a, w = np.abs(a), np.abs(w)
    p = np.zeros((a.shape[0], w.shape[0]))
    for j in range(0, a.shape[1], BLOCK):
        top = np.zeros_like(p)
        for k in range(j, min(j + BLOCK, a.shape[1])):
            np.maximum(top, np.outer(a[:, k], w[:, k]), out=top)
        p += top
    return p


def tolerance(y: np.ndarray, a: np.ndarray, w: np.ndarray) -> np.ndarray:
    """Bound of the matrix cores' sums (2**-10 of a block's largest product: the
    hardware aligns the products of an instruction and keeps about 15 bits below
    the largest, at most 2**-11.2 of it measured over 64 of them), of the fp32
    sums and of the bf16 output."""
    return (2.0 ** -10 * largest_products(a, w) + 1e-5 * (np.abs(a) @ np.abs(w).T)
            + 2.0 ** -8 * np.abs(y) + 2.0 ** -133)
