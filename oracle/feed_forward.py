"""Gated feed-forward and layer norm with their gradients, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Written from the
formulas; the gradients are pinned by differences of the forward forms.
"""

from __future__ import annotations

import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])


def activation(g: np.ndarray, act: str) -> np.ndarray:
    g = np.asarray(g, np.float64)
    if act == "silu":
        return g / (1 + np.exp(-g))
    if act == "gelu":
        return g * (1 + _erf(g / math.sqrt(2))) / 2
    return g * (1 + np.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))) / 2


def activation_slope(g: np.ndarray, act: str) -> np.ndarray:
    g = np.asarray(g, np.float64)
    if act == "silu":
        s = 1 / (1 + np.exp(-g))
        return s + g * s * (1 - s)
    if act == "gelu":
        return (1 + _erf(g / math.sqrt(2))) / 2 + g * np.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = np.tanh(c * (g + 0.044715 * g ** 3))
    return (1 + t) / 2 + g * (1 - t * t) / 2 * c * (1 + 3 * 0.044715 * g * g)


def gated(x, wg, wu, act):
    """(y, g, u)"""
    g, u = x @ wg.T, x @ wu.T
    return activation(g, act) * u, g, u


def gated_backward(dy, x, wg, wu, act):
    """(dx, dwg, dwu, dg, du)"""
    _, g, u = gated(x, wg, wu, act)
    dg, du = dy * u * activation_slope(g, act), dy * activation(g, act)
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x, dg, du


def layer_norm(x, w=None, b=None, eps=1e-5):
    """(y, mean, rstd)"""
    x = np.asarray(x, np.float64)
    mean = x.mean(axis=1, keepdims=True)
    rstd = 1 / np.sqrt(((x - mean) ** 2).mean(axis=1, keepdims=True) + eps)
    y = (x - mean) * rstd
    if w is not None:
        y = y * w
    return (y if b is None else y + b), mean, rstd


def layer_norm_backward(dy, x, w=None, eps=1e-5):
    """(dx, dw, db)"""
    h, _, rstd = layer_norm(x, eps=eps)
    t = dy if w is None else dy * w
    dx = rstd * (t - t.mean(axis=1, keepdims=True) - h * (t * h).mean(axis=1, keepdims=True))
    return dx, (dy * h).sum(axis=0), dy.sum(axis=0)
