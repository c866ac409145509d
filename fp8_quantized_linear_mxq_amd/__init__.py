"""Block-scaled (microscaling) quantized linear layers for AMD MI355X.

The compute lives in libmxq (HIP kernels for gfx950 behind the C ABI in
include/mxq.h); this package is its thin ctypes binding plus the seeded
synthetic workload generators.  Import is cheap: the library is loaded on
first use and its absence is an error, never a fallback.
"""
from ._lib import (  # noqa: F401
    ACTIVATIONS, BF16, DT_BF16, DT_F32, FORMATS, FP8, FP8_TILE, INT4, INT8, MXFP4, MXFP8, NVFP4, OP_GEMM, OP_LOWRANK_SPLIT,
    OP_GATED_BACKWARD, OP_LAYER_NORM_BACKWARD, OP_QUANTIZE, OP_QUANTIZE_MSE, OP_SELECT,
    MxqError, QTensor,
    act_format_for_step, bf16_operand, lowrank_split, conv3x3_gemm_mixed, empty_qtensor, gemm, gemm_grouped, gemm_mixed,
    fp8_operand, gemm_gated, gemm_gated_backward, int8_operand, layer_norm, layer_norm_backward, load,
    pack_l1t, qk_norm_rope, quantize, quantize_mse,
    select_format, storage, workspace_size,
)


def __getattr__(name):   # torch is imported with the differentiable functions only
    if name == "autograd":
        import importlib
        return importlib.import_module(".autograd", __name__)
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
