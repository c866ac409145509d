"""Operands whose codes or scales are one row, with the strides that torch gives them."""
import pytest
import torch

import fp8_quantized_linear_mxq_amd as mxq
from fp8_quantized_linear_mxq_amd import _lib


def test_row_strides_handed_to_the_library():
    codes = torch.zeros((5, 96), dtype=torch.uint8)
    scales = torch.ones((5, 1)).t().contiguous()     # [1, 5] with strides (1, 1)
    assert scales.stride(0) == 1
    c = mxq.fp8_operand(codes, scales).c()
    assert c.ld_codes == 96 and c.ld_scales >= 4 * 5 and c.ld_scales % 4 == 0
    c = mxq.fp8_operand(torch.zeros((300, 96), dtype=torch.uint8), torch.ones((3, 1)), tile=True).c()
    assert c.ld_scales == 4
    one = torch.zeros((96, 1), dtype=torch.uint8).t()   # a row of a transposed column
    c = mxq.fp8_operand(one, torch.ones((1, 1)), tile=True).c()
    assert c.ld_codes == 96 and c.ld_scales >= 4
    q = mxq.QTensor(_lib.MXFP4, 3, 64, torch.zeros((3, 48), dtype=torch.uint8)[:, :32], torch.zeros((3, 4), dtype=torch.uint8)).c()
    assert q.ld_codes == 48 and q.ld_scales == 4


@pytest.mark.gpu
@pytest.mark.parametrize("m,k", [(5, 96), (300, 128), (1, 320)])
def test_gemm_mixed(m, k):
    g = torch.Generator(device="cuda")
    g.manual_seed(m)
    w = torch.randint(-3, 4, (40, k), generator=g, device="cuda").float()
    a = torch.randint(-3, 4, (m, k), generator=g, device="cuda").float()
    kb = -(-k // 128)
    sa = torch.exp2(torch.randint(-1, 2, (m, kb), generator=g, device="cuda").float())
    qa = mxq.fp8_operand(a.to(torch.float8_e4m3fn), sa.t().contiguous())
    qw = mxq.fp8_operand(w.to(torch.float8_e4m3fn), torch.ones((1, kb), device="cuda"), tile=True)
    perm = torch.randperm(40, generator=g, device="cuda").int()
    want = torch.empty((m, 40), dtype=torch.bfloat16, device="cuda")
    want[:, perm.long()] = ((a * sa.repeat_interleave(128, 1)[:, :k]).double() @ w.double().t()).float().bfloat16()
    assert torch.equal(mxq.gemm_mixed(qa, [qw], perm, 40), want)
    assert torch.equal(mxq.gemm(qa, qw), want[:, perm.long()])
