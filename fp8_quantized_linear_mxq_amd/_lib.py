"""Binding of libmxq (include/mxq.h): ctypes, and for the calls that a model
makes in every layer (quantize, gemm, gemm_grouped, qk_norm_rope, gemm_gated,
layer_norm and their backward passes) the marshalling module built from csrc/torch_binding.cpp.

Argument marshalling only: every step of the layer runs inside libmxq's HIP
kernels.  PyTorch supplies device memory and the current stream.  If the
built library is missing, ``load()`` raises -- there is no fallback path.
"""
from __future__ import annotations

import ctypes as C
import os
from dataclasses import dataclass

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmxq.so")

MXFP4, MXFP8, NVFP4, INT4 = 1, 2, 3, 4
BF16 = 5   # unquantized bf16 activations (GEMM operand only)
INT8 = 6   # row-wise int8, one fp32 scale per row
FP8 = 7    # E4M3, one fp32 scale per row and 128 columns (activations)
FP8_TILE = 8   # E4M3, one fp32 scale per 128 x 128 tile (weights)
FORMATS = {"MXFP4": MXFP4, "MXFP8": MXFP8, "NVFP4": NVFP4, "INT4": INT4, "INT8": INT8, "FP8": FP8,
           "FP8_TILE": FP8_TILE}
FORMAT_NAMES = {v: k for k, v in FORMATS.items()}
DT_F32, DT_BF16 = 1, 2
OP_QUANTIZE, OP_GEMM, OP_SELECT, OP_QUANTIZE_MSE, OP_LOWRANK_SPLIT = 1, 2, 3, 4, 5
OP_GATED_BACKWARD, OP_LAYER_NORM_BACKWARD = 6, 7
BLOCK = {MXFP4: 32, MXFP8: 32, NVFP4: 16, INT4: 32}
ACTIVATIONS = {"silu": 1, "gelu": 2, "gelu_tanh": 3}

STATUS = {0: "MXQ_OK", 1: "MXQ_ERR_INVALID_ARG", 2: "MXQ_ERR_UNSUPPORTED",
          3: "MXQ_ERR_ALIGNMENT", 4: "MXQ_ERR_SHAPE", 5: "MXQ_ERR_WORKSPACE",
          6: "MXQ_ERR_NO_DEVICE", 7: "MXQ_ERR_LAUNCH", 8: "MXQ_ERR_NONFINITE"}

# Every symbol include/mxq.h declares.
EXPORTS = ("mxq_quantize", "mxq_quantize_noalloc", "mxq_quantize_lrp", "mxq_pack_l1t", "mxq_gemm", "mxq_gemm_mixed", "mxq_conv3x3_gemm_mixed",
           "mxq_gemm_grouped", "mxq_qk_norm_rope",
           "mxq_gemm_gated", "mxq_gemm_gated_backward", "mxq_layer_norm", "mxq_layer_norm_backward",
           "mxq_select_format", "mxq_quantize_mse", "mxq_lowrank_split",
           "mxq_act_format_for_step", "mxq_workspace_size", "mxq_storage",
           "mxq_status_string", "mxq_version")


class MxqError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {STATUS.get(status, status)}")
        self.status = status


class QTensorC(C.Structure):
    _fields_ = [("fmt", C.c_int32), ("reserved", C.c_int32),
                ("rows", C.c_int64), ("cols", C.c_int64),
                ("codes", C.c_void_p), ("ld_codes", C.c_int64),
                ("scales", C.c_void_p), ("ld_scales", C.c_int64),
                ("tensor_scale", C.c_void_p)]


_lib = None
_torch = None   # the torch module, bound by load(): an import statement costs 0.2 us a call
_fast = None    # the marshalling module


class _NotBuilt:
    """In place of the marshalling module: the calls through it raise, the
    library's other entry points work without it."""

    def __init__(self, cause):
        self.cause = cause

    def __getattr__(self, name):
        raise RuntimeError("the torch marshalling module is not built for this Python and torch; run "
                           "python -m fp8_quantized_linear_mxq_amd.build") from self.cause


def load():
    """Load libmxq.so (built in-tree by ``build.py``); raises if absent."""
    global _lib, _torch, _fast
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libmxq is not built ({LIB_PATH} missing); run "
                           "python -m fp8_quantized_linear_mxq_amd.build")
    try:  # share the HIP runtime torch already mapped (same soname)
        import torch
        _torch = torch
    except ImportError:
        pass
    lib = C.CDLL(LIB_PATH)
    vp, i32, i64, sz = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t
    qp = C.POINTER(QTensorC)
    lib.mxq_quantize.argtypes = [vp, i32, i64, i64, i64, i32, vp, vp, i32, vp, i64, qp, vp, sz, vp]
    lib.mxq_quantize.restype = i32
    lib.mxq_quantize_lrp.argtypes = [vp, i32, i64, i64, i64, i32, vp, vp, i32, vp, i64, qp, vp, sz, vp]
    lib.mxq_quantize_lrp.restype = i32
    lib.mxq_pack_l1t.argtypes = [vp, i32, i64, vp, vp]
    lib.mxq_pack_l1t.restype = i32
    lib.mxq_quantize_noalloc.argtypes = [vp, i32, i64, i64, i64, i32, vp, vp, i32, vp, i64, qp, vp]
    lib.mxq_quantize_noalloc.restype = i32
    lib.mxq_gemm.argtypes = [qp, qp, vp, vp, i64, vp, i32, vp, vp, i64, i64, vp, sz, vp]
    lib.mxq_gemm.restype = i32
    lib.mxq_gemm_mixed.argtypes = [qp, qp, i32, vp, vp, i64, vp, i32, vp, vp, i64, i64, vp, sz, vp]
    lib.mxq_gemm_mixed.restype = i32
    lib.mxq_gemm_grouped.argtypes = [qp, qp, i32, vp, vp, vp, i64, vp]
    lib.mxq_gemm_grouped.restype = i32
    lib.mxq_qk_norm_rope.argtypes = [vp, i32, i64, i64, i32, i32, i32, vp, vp, C.c_float, vp, vp, i64,
                                     i32, i32, vp, vp, i64, i64, vp, i64, i64, vp]
    lib.mxq_qk_norm_rope.restype = i32
    lib.mxq_gemm_gated.argtypes = [qp, qp, qp, i32, vp, vp, i64, vp]
    lib.mxq_gemm_gated.restype = i32
    lib.mxq_gemm_gated_backward.argtypes = [vp, i64, qp, qp, qp, i32, vp, vp, i64, vp, vp, i64, vp, sz, vp]
    lib.mxq_gemm_gated_backward.restype = i32
    lib.mxq_layer_norm.argtypes = [vp, i32, i64, i64, i64, vp, vp, C.c_float, vp, i64, vp, vp]
    lib.mxq_layer_norm.restype = i32
    lib.mxq_layer_norm_backward.argtypes = [vp, i64, vp, i32, i64, i64, i64, vp, vp, vp, i64, vp, vp, vp, sz, vp]
    lib.mxq_layer_norm_backward.restype = i32
    lib.mxq_conv3x3_gemm_mixed.argtypes = [qp, i64, i64, qp, i32, vp, vp, vp, i64, i64, vp, sz,
                                           vp]
    lib.mxq_conv3x3_gemm_mixed.restype = i32
    lib.mxq_select_format.argtypes = [vp, i32, i64, i64, i64, C.POINTER(i32), i32, vp, vp, vp,
                                      vp, vp, vp, sz, vp]
    lib.mxq_select_format.restype = i32
    lib.mxq_quantize_mse.argtypes = [vp, i32, i64, i64, i64, qp, vp, sz, vp]
    lib.mxq_quantize_mse.restype = i32
    lib.mxq_lowrank_split.argtypes = [vp, i64, i64, i64, i32, i32, vp, vp, vp, i64, vp, vp, sz, vp]
    lib.mxq_lowrank_split.restype = i32
    lib.mxq_act_format_for_step.argtypes = [C.POINTER(C.c_uint8), i32, i32, i32, i32, i32]
    lib.mxq_act_format_for_step.restype = i32
    lib.mxq_workspace_size.argtypes = [i32, i64, i64, i32]
    lib.mxq_workspace_size.restype = i64
    lib.mxq_storage.argtypes = [i32, i64, C.POINTER(i64), C.POINTER(i64)]
    lib.mxq_storage.restype = i32
    lib.mxq_status_string.argtypes = [i32]
    lib.mxq_status_string.restype = C.c_char_p
    lib.mxq_version.argtypes = []
    lib.mxq_version.restype = i32
    if _torch is not None:
        try:
            from . import _torch_binding
            _torch_binding.bind(*[C.cast(f, vp).value for f in (
                lib.mxq_quantize, lib.mxq_gemm, lib.mxq_gemm_grouped, lib.mxq_qk_norm_rope, lib.mxq_gemm_gated,
                lib.mxq_gemm_gated_backward, lib.mxq_layer_norm, lib.mxq_layer_norm_backward, lib.mxq_workspace_size)])
            _fast = _torch_binding
        except ImportError as e:
            _fast = _NotBuilt(e)
    _lib = lib
    return lib


def _check(fn: str, status: int):
    if status != 0:
        raise MxqError(fn, status)


def _ptr(t):
    return None if t is None else t.data_ptr()   # ctypes takes the integer


def _stream(stream):
    """The given stream's handle, or the current device's current stream (read
    as a handle: building the Stream object takes 3 us)."""
    if stream is not None:
        return stream.cuda_stream
    if _torch.cuda.is_initialized():
        return _torch._C._cuda_getCurrentRawStream(_torch._C._cuda_getDevice())
    return _torch.cuda.current_stream().cuda_stream if _torch.cuda.is_available() else 0


def _device(stream):
    """The device that the call's stream belongs to (-1 without a GPU: no tensor is on it)."""
    if stream is not None:
        return stream.device_index
    return _torch._C._cuda_getDevice() if _torch.cuda.is_initialized() else -1


def storage(fmt: int, cols: int):
    """(code bytes, scale bytes) per row for ``cols`` elements."""
    lib = load()
    cb, sb = C.c_int64(), C.c_int64()
    _check("mxq_storage", lib.mxq_storage(fmt, cols, C.byref(cb), C.byref(sb)))
    return cb.value, sb.value


def workspace_size(op: int, rows: int, cols: int, fmt: int = 0) -> int:
    return int(load().mxq_workspace_size(op, rows, cols, fmt))


def act_format_for_step(table, n_layers: int, n_buckets: int, layer: int, step: int,
                        num_steps: int) -> int:
    lib = load()
    buf = (C.c_uint8 * len(table))(*[int(v) for v in table])
    return int(lib.mxq_act_format_for_step(buf, n_layers, n_buckets, layer, step, num_steps))


def _row_bytes(t, align: int) -> int:
    """Bytes between rows.  A single row may have any stride in torch (that of a
    transposed column is 1): one that the library would refuse is replaced."""
    given = t.stride(0) * t.element_size()
    if len(t) != 1:
        return given
    width = t.numel() * t.element_size()
    return given if given >= width and given % align == 0 else (width + 15) // 16 * 16


@dataclass
class QTensor:
    """A quantized [rows, cols] operand in device memory (torch uint8 / fp32)."""
    fmt: int
    rows: int
    cols: int
    codes: "object"
    scales: "object"
    tensor_scale: "object" = None

    def c(self) -> QTensorC:
        codes, scales, ts = self.codes, self.scales, self.tensor_scale
        return QTensorC(self.fmt, 0, self.rows, self.cols,
                        codes.data_ptr() if codes is not None else None,
                        _row_bytes(codes, 16) if codes is not None else 0,
                        scales.data_ptr() if scales is not None else None,
                        _row_bytes(scales, 16 if self.fmt == INT4 else 4) if scales is not None else 0,
                        ts.data_ptr() if ts is not None else None)


def empty_qtensor(fmt: int, rows: int, cols: int, device="cuda") -> QTensor:
    """Allocates (torch) the buffers of a quantized operand."""
    import torch
    cb, sb = storage(fmt, cols)
    # row strides padded to the ABI's alignment (16 B codes; 4 B scales, 16 B
    # for INT4's fp32 scales)
    codes = torch.empty((rows, (cb + 15) // 16 * 16), dtype=torch.uint8, device=device)
    if fmt == INT8:
        scales = torch.empty((rows, 1), dtype=torch.float32, device=device)
    elif fmt in (FP8, FP8_TILE):   # K-blocks of all rows, or tiles
        shape = (sb // 4, rows) if fmt == FP8 else ((rows + 127) // 128, sb // 4)
        scales = torch.empty(shape, dtype=torch.float32, device=device)
    elif fmt == INT4:
        scales = torch.empty((rows, (sb // 4 + 3) // 4 * 4), dtype=torch.float32, device=device)
    else:
        scales = torch.empty((rows, (sb + 3) // 4 * 4), dtype=torch.uint8, device=device)
    ts = torch.empty((1,), dtype=torch.float32, device=device) if fmt == NVFP4 else None
    return QTensor(fmt, rows, cols, codes, scales, ts)


def bf16_operand(x) -> QTensor:
    """A 2-D cuda bfloat16 tensor as the GEMM's unquantized activation
    operand (4-bit weights, 16-bit activations)."""
    import torch
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("bf16_operand needs a row-major 2-D bfloat16 tensor")
    return QTensor(BF16, x.shape[0], x.shape[1], x, None)


def int8_operand(codes, scales) -> QTensor:
    """int8 codes [rows, K] (cuda, row-major; int8, or their bits as uint8)
    and one float32 scale per row ([rows] or [rows, 1]) as a quantized operand."""
    shape = codes.shape
    if len(shape) != 2 or codes.element_size() != 1 or codes.is_floating_point() or \
            (codes.stride(1) != 1 and shape[1] > 1):
        raise ValueError("int8_operand needs row-major 2-D 8-bit integer codes")
    rows, cols = shape
    sshape = scales.shape
    if scales.element_size() != 4 or not scales.is_floating_point() or sshape[0] != rows or \
            not (len(sshape) == 1 or (len(sshape) == 2 and sshape[1] == 1)):
        raise ValueError("int8_operand needs float32 scales of shape [rows] or [rows, 1]")
    return QTensor(INT8, rows, cols, codes, scales)


_E4M3_TYPES = ("torch.float8_e4m3fn", "torch.uint8", "torch.int8")   # int8: their bits


def fp8_operand(codes, scales, tile: bool = False) -> QTensor:
    """E4M3 codes [rows, K] (cuda, row-major; float8_e4m3fn, or their bits as
    uint8) as a quantized operand: activations with float32 scales
    [ceil(K / 128), rows], or with ``tile`` weights with scales
    [ceil(rows / 128), ceil(K / 128)]; rows of the scales contiguous."""
    shape = codes.shape
    if len(shape) != 2 or str(codes.dtype) not in _E4M3_TYPES or \
            (codes.stride(1) != 1 and shape[1] > 1):
        raise ValueError("fp8_operand needs row-major 2-D E4M3 codes")
    rows, cols = shape
    kb = (cols + 127) // 128
    want = ((rows + 127) // 128, kb) if tile else (kb, rows)
    if scales.element_size() != 4 or not scales.is_floating_point() or scales.shape != want or \
            (scales.stride(1) != 1 and want[1] > 1):
        raise ValueError(f"fp8_operand needs float32 scales of shape {list(want)}")
    return QTensor(FP8_TILE if tile else FP8, rows, cols, codes, scales)


def pack_l1t(l1t, stream=None):
    """mxq_pack_l1t: L1^T [rank, cols] bf16 (cuda) into the packed order the
    fused quantize + low-rank kernel reads; returned with the same shape."""
    import torch
    lib = load()
    if stream is not None:   # what is allocated here belongs to the stream that writes it
        with torch.cuda.stream(stream):
            return pack_l1t(l1t)
    rank, cols = l1t.shape
    l1t = l1t.contiguous()
    out = torch.empty_like(l1t)
    _check("mxq_pack_l1t", lib.mxq_pack_l1t(_ptr(l1t), rank, cols, _ptr(out), _stream(None)))
    return out


def quantize(x, fmt: int, hadamard: int = 0, static_tensor_scale=None, l1t=None, u=None,
             out: QTensor | None = None, workspace=None, stream=None, l1p=None) -> QTensor:
    """mxq_quantize on a 2-D torch tensor (float32 or bfloat16, cuda); with
    ``l1p`` (L1 from pack_l1t) instead of ``l1t``, mxq_quantize_lrp."""
    lib = load()
    torch = _torch
    if stream is not None and (out is None or workspace is None):
        with torch.cuda.stream(stream):   # what is allocated here belongs to the stream that writes it
            return quantize(x, fmt, hadamard, static_tensor_scale, l1t, u, out, workspace, l1p=l1p)
    rows, cols = x.shape
    dt = DT_BF16 if x.dtype == torch.bfloat16 else DT_F32
    if out is None:
        out = (QTensor(fmt, rows, cols, *_fast.empty_rows(x, fmt)) if fmt in (INT8, FP8, FP8_TILE) and cols % 32 == 0
               else empty_qtensor(fmt, rows, cols, x.device))
    if workspace is None:
        n = workspace_size(OP_QUANTIZE, rows, cols, fmt) if fmt == NVFP4 else 0   # the one that needs any
        if n > 0:
            workspace = torch.empty((n,), dtype=torch.uint8, device=x.device)
    wsn = 0 if workspace is None else workspace.numel()
    if l1p is not None:
        qc = out.c()
        st = lib.mxq_quantize_lrp(_ptr(x), dt, rows, cols, x.stride(0), hadamard,
                                  _ptr(static_tensor_scale), _ptr(l1p), l1p.shape[0], _ptr(u),
                                  0 if u is None else u.stride(0), C.byref(qc), _ptr(workspace), wsn,
                                  _stream(stream))
        _check("mxq_quantize_lrp", st)
        return out
    st = _fast.quantize(x, dt, hadamard, static_tensor_scale, l1t, u, out, workspace, wsn, _stream(stream))
    if st != 0:
        raise MxqError("mxq_quantize", st)
    return out


def _gemm_workspace(a: QTensor, ws: list, workspace):
    """The optional GEMM workspace: a given tensor, none (workspace=False),
    or a fresh one sized for the largest of the weight operands ``ws``."""
    import torch
    if workspace is False:
        return None, 0
    if workspace is None:
        # only INT4 weights can use one
        if all(w.fmt != INT4 for w in ws):
            return None, 0
        n = max([workspace_size(OP_GEMM, a.rows, w.rows, w.fmt) for w in ws] + [0])
        if n <= 0:
            return None, 0
        workspace = torch.empty((n,), dtype=torch.uint8, device=a.codes.device)
    return _ptr(workspace), workspace.numel() * workspace.element_size()


def gemm(a: QTensor, w: QTensor, n_out: int | None = None, w_out_col=None, u=None, l2t=None,
         bias=None, out=None, stream=None, workspace=None):
    """mxq_gemm; returns the bf16 [M, n_out] output tensor.  ``workspace``:
    a device tensor, None (allocated when the route can use one) or False."""
    load()
    if stream is not None and (out is None or workspace is None):
        with _torch.cuda.stream(stream):
            return gemm(a, w, n_out, w_out_col, u, l2t, bias, out, workspace=workspace)
    wsn = 0
    if workspace is False:
        workspace = None
    elif workspace is not None:
        wsn = workspace.numel() * workspace.element_size()
    elif w.fmt == INT4:   # the one weight format that can use one
        wsn = workspace_size(OP_GEMM, a.rows, w.rows, w.fmt)
        if wsn > 0:
            workspace = _torch.empty((wsn,), dtype=_torch.uint8, device=a.codes.device)
        wsn = max(wsn, 0)
    r = _fast.gemm(a, w, w.rows if n_out is None else n_out, w_out_col, u, l2t, bias, out, workspace, wsn,
                   _stream(stream))
    if type(r) is int:
        raise MxqError("mxq_gemm", r)
    return r


def gemm_mixed(a: QTensor, groups: list, w_perm, n_out: int, u=None, l2t=None, bias=None,
               out=None, stream=None, workspace=None):
    """mxq_gemm_mixed over weight groups (QTensor list) and their permutation."""
    import torch
    lib = load()
    if stream is not None:   # what is allocated here belongs to the stream that writes it
        with torch.cuda.stream(stream):
            return gemm_mixed(a, groups, w_perm, n_out, u, l2t, bias, out, workspace=workspace)
    if out is None:
        out = torch.empty((a.rows, n_out), dtype=torch.bfloat16, device=a.codes.device)
    ac = a.c()
    arr = (QTensorC * len(groups))(*[g.c() for g in groups])
    rank = 0 if l2t is None else l2t.shape[1]
    wsp, wsn = _gemm_workspace(a, groups, workspace)
    st = lib.mxq_gemm_mixed(C.byref(ac), arr, len(groups), _ptr(w_perm), _ptr(u),
                            0 if u is None else u.stride(0), _ptr(l2t), rank, _ptr(bias),
                            _ptr(out), out.stride(0), n_out, wsp, wsn, _stream(None))
    _check("mxq_gemm_mixed", st)
    return out


def gemm_grouped(a: QTensor, w: QTensor, offsets, bias=None, out=None, stream=None):
    """mxq_gemm_grouped: rows of ``a`` sorted by expert, ``offsets`` (int32,
    cuda, [experts + 1]) their groups, ``w`` the experts' weights one after
    the other ([experts * N, K]), ``bias`` bf16 [experts, N]; returns the bf16
    [rows, N] output tensor (rows of no group are left as they are in ``out``)."""
    load()
    if stream is not None and out is None:
        with _torch.cuda.stream(stream):
            return gemm_grouped(a, w, offsets, bias)
    r = _fast.gemm_grouped(a, w, offsets, bias, out, _stream(stream))
    if type(r) is int:
        raise MxqError("mxq_gemm_grouped", r)
    return r


def qk_norm_rope(x, n_q_heads: int, n_k_heads: int, head_dim: int, q_weight=None, k_weight=None,
                 cos=None, sin=None, positions=None, eps: float = 1e-6, interleaved: bool = False,
                 q_out=None, k_out=None, stream=None):
    """mxq_qk_norm_rope on the 2-D output of a fused projection (float32 or
    bfloat16, cuda): RMS norm of every query and key head and the position
    rotation given by the float32 tables ``cos`` and ``sin`` [n_pos, rot/2].
    Returns (q [tokens, n_q_heads, head_dim], k [tokens, n_k_heads, head_dim]);
    ``q_out`` and ``k_out`` may be given with any token and head strides."""
    load()
    if stream is not None and (q_out is None or k_out is None):
        with _torch.cuda.stream(stream):
            return qk_norm_rope(x, n_q_heads, n_k_heads, head_dim, q_weight, k_weight, cos, sin, positions,
                                eps, interleaved, q_out, k_out)
    r = _fast.qk_norm_rope(x, n_q_heads, n_k_heads, head_dim, q_weight, k_weight, cos, sin, positions,
                           eps, int(interleaved), q_out, k_out, _stream(stream))
    if type(r) is int:
        raise MxqError("mxq_qk_norm_rope", r)
    return r


def gemm_gated(x: QTensor, w_gate: QTensor, w_up: QTensor, act: str = "silu", saved=None, out=None, stream=None):
    """mxq_gemm_gated: bf16 [rows, N] of act(x w_gate^T) * (x w_up^T), ``act``
    one of ACTIVATIONS, on FP8 activations and FP8_TILE weights or on bf16
    operands (bf16_operand).  ``saved``: a float32 tensor [2, rows, N] that
    receives both products for gemm_gated_backward (bf16 only)."""
    load()
    if stream is not None and out is None:
        with _torch.cuda.stream(stream):
            return gemm_gated(x, w_gate, w_up, act, saved)
    r = _fast.gemm_gated(x, w_gate, w_up, ACTIVATIONS.get(act, 0), saved, out, _device(stream), _stream(stream))
    if type(r) is int:
        raise MxqError("mxq_gemm_gated", r)
    return r


def gemm_gated_backward(dy, x: QTensor, w_gate: QTensor, w_up: QTensor, saved, act: str = "silu", dx=None,
                        dw_gate=None, dw_up=None, want=(True, True), workspace=None, stream=None):
    """mxq_gemm_gated_backward: (dx, dw_gate, dw_up) of gemm_gated on bf16
    operands for the bf16 gradient ``dy`` [rows, N]; ``want``: whether dx and
    the weights' gradients are formed (None in their place otherwise)."""
    load()
    if stream is not None:   # what is allocated here belongs to the stream that writes it
        with _torch.cuda.stream(stream):
            return gemm_gated_backward(dy, x, w_gate, w_up, saved, act, dx, dw_gate, dw_up, want, workspace)
    r = _fast.gemm_gated_backward(dy, x, w_gate, w_up, ACTIVATIONS.get(act, 0), saved, int(want[0]), int(want[1]),
                                  dx, dw_gate, dw_up, workspace, _device(None), _stream(None))
    if type(r) is int:
        raise MxqError("mxq_gemm_gated_backward", r)
    return r


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, stats=None, out=None, stream=None):
    """mxq_layer_norm over the rows of a 2-D tensor (float32 or bfloat16,
    cuda), ``weight`` and ``bias`` [cols] of its dtype.  ``stats``: a float32
    tensor [rows, 2] that receives each row's mean and reciprocal deviation
    for layer_norm_backward."""
    load()
    if stream is not None and out is None:
        with _torch.cuda.stream(stream):
            return layer_norm(x, weight, bias, eps, stats)
    r = _fast.layer_norm(x, weight, bias, eps, stats, out, _device(stream), _stream(stream))
    if type(r) is int:
        raise MxqError("mxq_layer_norm", r)
    return r


def layer_norm_backward(dy, x, stats, weight=None, want=(True, True), dx=None, dweight=None, dbias=None,
                        workspace=None, stream=None):
    """mxq_layer_norm_backward: (dx, dweight, dbias) for the gradient ``dy`` of
    layer_norm's output; ``want``: whether dx and the parameters' gradients
    are formed (None in their place otherwise)."""
    load()
    if stream is not None:   # what is allocated here belongs to the stream that writes it
        with _torch.cuda.stream(stream):
            return layer_norm_backward(dy, x, stats, weight, want, dx, dweight, dbias, workspace)
    r = _fast.layer_norm_backward(dy, x, stats, weight, int(want[0]), int(want[1]), dx, dweight, dbias, workspace,
                                  _device(None), _stream(None))
    if type(r) is int:
        raise MxqError("mxq_layer_norm_backward", r)
    return r


def conv3x3_gemm_mixed(x: QTensor, height: int, width: int, groups: list, w_perm, n_out: int,
                       bias=None, out=None, stream=None, workspace=None):
    """mxq_conv3x3_gemm_mixed: the 3x3 convolution (stride 1, zero padding 1)
    of the quantized pixel rows ``x`` ([images*height*width, C]) with weight
    groups of 9*C columns; returns the bf16 [x.rows, n_out] output tensor."""
    import torch
    lib = load()
    if stream is not None:   # what is allocated here belongs to the stream that writes it
        with torch.cuda.stream(stream):
            return conv3x3_gemm_mixed(x, height, width, groups, w_perm, n_out, bias, out, workspace=workspace)
    if out is None:
        out = torch.empty((x.rows, n_out), dtype=torch.bfloat16, device=x.codes.device)
    xc = x.c()
    arr = (QTensorC * len(groups))(*[g.c() for g in groups])
    wsp, wsn = _gemm_workspace(x, groups, workspace)
    st = lib.mxq_conv3x3_gemm_mixed(C.byref(xc), height, width, arr, len(groups), _ptr(w_perm),
                                    _ptr(bias), _ptr(out), out.stride(0), n_out, wsp, wsn,
                                    _stream(None))
    _check("mxq_conv3x3_gemm_mixed", st)
    return out


def select_format(w, candidates=(INT4, MXFP4, NVFP4), stream=None):
    """mxq_select_format; returns (choice u8[n], sse f64[n, c], perm i32[n],
    counts i32[c], g f32[1]) as device tensors."""
    import torch
    lib = load()
    if stream is not None:   # what is allocated here belongs to the stream that writes it
        with torch.cuda.stream(stream):
            return select_format(w, candidates)
    n, k = w.shape
    dt = DT_BF16 if w.dtype == torch.bfloat16 else DT_F32
    dev = w.device
    choice = torch.empty((n,), dtype=torch.uint8, device=dev)
    sse = torch.empty((n, len(candidates)), dtype=torch.float64, device=dev)
    perm = torch.empty((n,), dtype=torch.int32, device=dev)
    counts = torch.empty((len(candidates),), dtype=torch.int32, device=dev)
    g = torch.empty((1,), dtype=torch.float32, device=dev)
    ws = torch.empty((workspace_size(OP_SELECT, n, k),), dtype=torch.uint8, device=dev)
    cand = (C.c_int32 * len(candidates))(*candidates)
    st = lib.mxq_select_format(_ptr(w), dt, n, k, w.stride(0), cand, len(candidates),
                               _ptr(choice), _ptr(sse), _ptr(perm), _ptr(counts), _ptr(g),
                               _ptr(ws), ws.numel(), _stream(None))
    _check("mxq_select_format", st)
    return choice, sse, perm, counts, g


def quantize_mse(w, fmt: int, out: QTensor | None = None, workspace=None,
                 stream=None) -> QTensor:
    """mxq_quantize_mse on 2-D torch weights (float32 or bfloat16, cuda):
    MXFP4 or NVFP4 codes with least-squared-error scales."""
    import torch
    lib = load()
    if stream is not None:   # what is allocated here belongs to the stream that writes it
        with torch.cuda.stream(stream):
            return quantize_mse(w, fmt, out, workspace)
    rows, cols = w.shape
    dt = DT_BF16 if w.dtype == torch.bfloat16 else DT_F32
    if out is None:
        out = empty_qtensor(fmt, rows, cols, w.device)
    if workspace is None:
        n = workspace_size(OP_QUANTIZE_MSE, rows, cols, fmt)
        workspace = torch.empty((max(n, 16),), dtype=torch.uint8, device=w.device)
    qc = out.c()
    st = lib.mxq_quantize_mse(_ptr(w), dt, rows, cols, w.stride(0), C.byref(qc),
                              _ptr(workspace), workspace.numel(), _stream(None))
    _check("mxq_quantize_mse", st)
    return out


def lowrank_split(w, rank: int, iters: int = 0, stream=None):
    """mxq_lowrank_split on 2-D float32 cuda weights [n, k]; returns
    (L1^T bf16 [rank, k], L2^T bf16 [n, rank], R float32 [n, k],
    sigma float32 [rank])."""
    import torch
    lib = load()
    if stream is not None:   # what is allocated here belongs to the stream that writes it
        with torch.cuda.stream(stream):
            return lowrank_split(w, rank, iters)
    n, k = w.shape
    dev = w.device
    l1t = torch.empty((rank, k), dtype=torch.bfloat16, device=dev)
    l2t = torch.empty((n, rank), dtype=torch.bfloat16, device=dev)
    resid = torch.empty((n, k), dtype=torch.float32, device=dev)
    sigma = torch.empty((rank,), dtype=torch.float32, device=dev)
    ws = torch.empty((max(workspace_size(OP_LOWRANK_SPLIT, n, k, rank), 256),),
                     dtype=torch.uint8, device=dev)
    st = lib.mxq_lowrank_split(_ptr(w), n, k, w.stride(0), rank, iters, _ptr(l1t), _ptr(l2t),
                               _ptr(resid), resid.stride(0), _ptr(sigma), _ptr(ws), ws.numel(),
                               _stream(None))
    _check("mxq_lowrank_split", st)
    return l1t, l2t, resid, sigma
