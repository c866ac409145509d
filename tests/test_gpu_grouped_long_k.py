"""Long sums of the products grouped by expert: the bound of every GEMM route
has to hold where one fp32 chain over all of K would break it."""
import numpy as np
import pytest

from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


def _ones(rows, k):
    """MXFP4 weights of 1."""
    import torch
    import fp8_quantized_linear_mxq_amd as mxq
    return mxq.QTensor(mxq.MXFP4, rows, k, torch.full((rows, k // 2), 0x22, dtype=torch.uint8, device="cuda"),
                       torch.full((rows, k // 32), 127, dtype=torch.uint8, device="cuda"))


def _large_then_small(pair, k, larges):
    """An activation row with 2**25 at the given places and 1.5, below half of
    its last place in fp32, at one K of each further matrix instruction (every
    8th of the first 32 in a run of 128 for bf16, the first for MXFP4): (operand,
    exact sum over the small ones, how many large ones)."""
    import torch
    import fp8_quantized_linear_mxq_amd as mxq
    if pair == "BF16":
        a = torch.zeros(1, k)
        a.view(-1, 128)[:, 0:32:8] = 1.5
        a[0, larges] = 2.0 ** 25
        return mxq.bf16_operand(a.bfloat16().cuda()), float(a[a == 1.5].double().sum())
    codes = torch.zeros(1, k // 2, dtype=torch.uint8)
    scales = torch.full((1, k // 32), 127, dtype=torch.uint8)
    codes[0, ::64] = 3                                         # 1.5
    for p in larges:
        codes[0, p // 2], scales[0, p // 32] = 6, 127 + 23     # 4 * 2**23
    return mxq.QTensor(mxq.MXFP4, 1, k, codes.cuda(), scales.cuda()), 1.5 * int((codes == 3).sum())


@pytest.mark.parametrize("pair,k", [("BF16", 65536), ("BF16", 262144), ("MXFP4", 262144), ("MXFP4", 786432)])
def test_few_rows_small_after_large(pair, k):
    """A large product at the head of each wave's share, small ones after it,
    and a bias that takes the large ones away again.  The bound is that of every
    route, with S the sum of the products."""
    import torch
    import fp8_quantized_linear_mxq_amd as mxq
    gu.say(f"grouped {pair} few rows K={k}")
    larges = [256 * w for w in range(4)]
    a, small = _large_then_small(pair, k, larges)
    bias = torch.full((2, 20), -float(len(larges)) * 2.0 ** 25, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 0, 1], dtype=torch.int32, device="cuda")
    y = mxq.gemm_grouped(a, _ones(40, k), off, bias=bias).double().cpu().numpy()
    s = len(larges) * 2.0 ** 25 + small
    tol = 1e-5 * (1 + 2 ** -8) * s + 2.0 ** -8 * small
    assert np.all(np.abs(y - small) <= tol), f"got {np.unique(y)}, exact {small}, bound {tol:.4g}"


@pytest.mark.parametrize("pair", ["BF16", "MXFP4"])
@pytest.mark.parametrize("k", [4224, 8320, 12416])
def test_few_rows_several_rounds(pair, k):
    """Ragged sizes over the second and third round of the K loop."""
    from tests.test_gpu_grouped import _check
    _check(pair, [1, 0, 17, 3], 45, k, seed=k, bias=True)
    _check(pair, [2] * 5, 33, k, seed=k + 1)
