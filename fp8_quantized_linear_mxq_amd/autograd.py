"""The operators with gradients as differentiable torch functions.

Both run the library's own forward and backward kernels; torch only keeps what
the backward pass needs and hands it over.  Leading dimensions are kept: the
last one is the operator's row.  Gradients of gradients are not formed.

In a captured graph call the library's functions themselves (gemm_gated and
gemm_gated_backward, layer_norm and layer_norm_backward): autograd ties the
gradients of a leaf to the stream on which it was first used, and a captured
backward pass that waits for another stream ends the process.  With a gradient
to form, the functions here refuse to run in a capture (RuntimeError).
"""
from __future__ import annotations

import torch

from . import _lib


def _rows(t):
    """t as a row-major matrix of its last dimension."""
    cols = t.shape[-1]
    t = t.reshape(t.numel() // max(1, cols), cols)
    return t if t.stride(1) == 1 and t.stride(0) >= cols else t.contiguous()


def _no_capture(names):
    if torch.cuda.is_current_stream_capturing():
        raise RuntimeError(f"gradients in a captured graph are formed with {names}, not through autograd")


def _keeps(names, *tensors):
    """Whether the call is one to differentiate."""
    keep = torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)
    if keep:
        _no_capture(names)
    return keep


class _Gated(torch.autograd.Function):
    names = "gemm_gated and gemm_gated_backward"

    @staticmethod
    def forward(ctx, x, w_gate, w_up, act, keep):
        x2 = _rows(x)
        ops = [_lib.bf16_operand(t) for t in (x2, w_gate, w_up)]
        saved = None
        if keep:
            saved = torch.empty((2, x2.shape[0], w_gate.shape[0]), dtype=torch.float32, device=x.device)
        y = _lib.gemm_gated(*ops, act=act, saved=saved)
        ctx.save_for_backward(x2, w_gate, w_up, saved)
        ctx.act, ctx.shape = act, x.shape
        return y.view(*x.shape[:-1], w_gate.shape[0])

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        _no_capture(_Gated.names)
        x, w_gate, w_up, saved = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dwg, dwu = _lib.gemm_gated_backward(_rows(dy), *(_lib.bf16_operand(t) for t in (x, w_gate, w_up)), saved,
                                                act=ctx.act, want=(need[0], need[1] or need[2]))
        return (None if dx is None else dx.view(ctx.shape), dwg if need[1] else None, dwu if need[2] else None, None, None)


def gated(x, w_gate, w_up, act: str = "silu"):
    """act(x w_gate^T) * (x w_up^T) of bfloat16 x [..., K] and weights [N, K]
    (rows at 16-byte alignment), with gradients for all three."""
    return _Gated.apply(x, w_gate, w_up, act, _keeps(_Gated.names, x, w_gate, w_up))


class _LayerNorm(torch.autograd.Function):
    names = "layer_norm and layer_norm_backward"

    @staticmethod
    def forward(ctx, x, weight, bias, eps, keep):
        x2 = _rows(x)
        stats = None
        if keep:
            stats = torch.empty((x2.shape[0], 2), dtype=torch.float32, device=x.device)
        y = _lib.layer_norm(x2, weight, bias, eps=eps, stats=stats)
        ctx.save_for_backward(x2, weight, stats)
        ctx.shape = x.shape
        return y.view(x.shape)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        _no_capture(_LayerNorm.names)
        x, weight, stats = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw, db = _lib.layer_norm_backward(_rows(dy), x, stats, weight, want=(need[0], need[1] or need[2]))
        return (None if dx is None else dx.view(ctx.shape), dw if need[1] else None, db if need[2] else None, None, None)


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5):
    """Norm over the last dimension of float32 or bfloat16 x, weight and bias of
    its dtype, with gradients for all three."""
    return _LayerNorm.apply(x, weight, bias, eps, _keeps(_LayerNorm.names, x, weight, bias))
