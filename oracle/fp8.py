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
    """The contract's bound (below) with only a block's largest product in place of
    that of every eight: closer, and enough for data whose large products do not
    lie next to many small ones of one sign."""
    return (2.0 ** -10 * largest_products(a, w) + 1e-5 * (np.abs(a) @ np.abs(w).T)
            + 2.0 ** -8 * np.abs(y) + 2.0 ** -133)


def largest_of_eight(ca: np.ndarray, sa: np.ndarray, cw: np.ndarray, sw: np.ndarray) -> np.ndarray:
    """Q [M, N]: over the groups of eight consecutive k, the sum of the largest |a w| of
    each, codes below E4M3's smallest normal counted as that."""
    up = lambda c, s, t: np.maximum(np.abs(E4M3.decode(c)), 2.0 ** -6) * spread(s, *c.shape, t)   # noqa: E731
    a, w = up(ca, sa, False), up(cw, sw, True)
    q = np.zeros((a.shape[0], w.shape[0]))
    for j in range(0, a.shape[1], 8):
        top = np.outer(a[:, j], w[:, j])
        for k in range(j + 1, j + 8):
            np.maximum(top, np.outer(a[:, k], w[:, k]), out=top)
        q += top
    return q


def bound(ca: np.ndarray, sa: np.ndarray, cw: np.ndarray, sw: np.ndarray) -> np.ndarray:
    """The contract's bound of a product of codes.  The matrix instruction takes eight
    consecutive k together and cuts each product to a multiple of 2**-13 of the
    group's leading binade: seven of them lose less than 7 * 2**-13 < 2**-10 of its
    largest.  Then the fp32 sums and the bf16 output."""
    a, w = dequantize(ca, sa), dequantize(cw, sw, True)
    sums = max(1e-5, 2.0 ** -30 * a.shape[1])
    return (2.0 ** -10 * largest_of_eight(ca, sa, cw, sw) + sums * (np.abs(a) @ np.abs(w).T)
            + 2.0 ** -8 * np.abs(a @ w.T) + 2.0 ** -133)
