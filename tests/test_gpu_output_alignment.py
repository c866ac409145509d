"""Output rows of every alignment: the same bits as in 16-byte aligned rows,
and nothing beside them, for the stores of each product's route."""
import pytest
import torch

import fp8_quantized_linear_mxq_amd as mxq
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

PAIRS = {"mxfp4": (mxq.MXFP4, mxq.MXFP4), "nvfp4": (mxq.NVFP4, mxq.NVFP4), "mxfp8 x nvfp4": (mxq.MXFP8, mxq.NVFP4),
         "bf16 x mxfp4": (mxq.BF16, mxq.MXFP4), "mxfp8 x mxfp4": (mxq.MXFP8, mxq.MXFP4),
         "mxfp8 x int4": (mxq.MXFP8, mxq.INT4), "int8": (mxq.INT8, mxq.INT8)}


def _operand(x, fmt):
    return mxq.bf16_operand(x.bfloat16()) if fmt == mxq.BF16 else mxq.quantize(x, fmt)


# rows and columns that end inside tiles and inside 8-, 4- and 2-element pieces;
# small and large tiles, and K past the slabs' threshold
@pytest.mark.parametrize("m,n,k", [(33, 77, 256), (300, 262, 384), (70, 131, 4352), (2100, 4100, 256), (1000, 6151, 128)])
@pytest.mark.parametrize("pair", PAIRS)
def test_rows_of_any_alignment(pair, m, n, k):
    gu.say(f"{pair} {m}x{n}x{k} into rows of every alignment")
    g = torch.Generator(device="cuda")
    g.manual_seed(m + n)
    fa, fw = PAIRS[pair]
    a = _operand(torch.randn(m, k, generator=g, device="cuda"), fa)
    w = mxq.quantize(torch.randn(n, k, generator=g, device="cuda"), fw)
    bias = torch.randn(n, generator=g, device="cuda").bfloat16()
    w8 = (n + 15) // 8 * 8
    want = torch.full((m, w8), -7.0, dtype=torch.bfloat16, device="cuda")
    mxq.gemm(a, w, bias=bias, out=want)
    grouped = (fa, fw) in ((mxq.MXFP4, mxq.MXFP4), (mxq.BF16, mxq.MXFP4), (mxq.INT8, mxq.INT8))
    off = torch.tensor([0, m], dtype=torch.int32, device="cuda")
    if grouped:
        want_g = torch.full((m, w8), -7.0, dtype=torch.bfloat16, device="cuda")
        mxq.gemm_grouped(a, w, off, bias=bias, out=want_g)
    for stride in (w8, w8 + 4, w8 + 2, w8 + 1):
        for first in (0, 4, 2, 1):       # elements past a 16-byte boundary
            def check(call, want):
                flat = torch.full((first + (m + 1) * stride,), -7.0, dtype=torch.bfloat16, device="cuda")
                call(flat[first:].view(m + 1, stride)[:m])
                rows = flat[first:].view(m + 1, stride)
                assert torch.equal(rows[:m, :n], want[:, :n]), (stride % 8, first)
                assert bool((rows[:m, n:] == -7).all()) and bool((rows[m] == -7).all()) and bool((flat[:first] == -7).all())
            check(lambda out: mxq.gemm(a, w, bias=bias, out=out), want)
            if grouped:
                check(lambda out: mxq.gemm_grouped(a, w, off, bias=bias, out=out), want_g)
