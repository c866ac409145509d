"""NaN in the gated products and their gradients: what the formulas give, and nothing in
rows and columns beside them."""
import pytest
import torch

import fp8_quantized_linear_mxq_amd as mxq
from tests.test_gpu_gated import exact_case

pytestmark = pytest.mark.gpu

ACTS = ["silu", "gelu", "gelu_tanh"]
NAN = float("nan")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n", [(40, 64), (40, 51)])   # eight columns and two columns to a thread
def test_nan_gate(m, n, act):
    """A NaN gate makes its outputs' gradients NaN: f'(g) is."""
    x, wg, wu, dy, gate, up = exact_case(m, n, 64)
    ops = [mxq.bf16_operand(t.bfloat16()) for t in (x, wg, wu)]
    saved = torch.stack([gate, up]).float()
    clean = mxq.gemm_gated_backward(dy.bfloat16(), *ops, saved, act=act)
    saved[0, 7, 5] = NAN
    dx, dwg, dwu = mxq.gemm_gated_backward(dy.bfloat16(), *ops, saved, act=act)
    assert bool(dx[7].isnan().all()) and bool(dwg[5].isnan().all()) and bool(dwu[5].isnan().all())
    rows, outs = torch.arange(m, device="cuda") != 7, torch.arange(n, device="cuda") != 5
    assert torch.equal(dx[rows], clean[0][rows])
    assert torch.equal(dwg[outs], clean[1][outs]) and torch.equal(dwu[outs], clean[2][outs])


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m", [3, 200])   # few rows, tiles
def test_nan_input(m, act):
    """A NaN of x reaches its row of the outputs and of the pre-activations, and no other."""
    x, wg, wu, dy, gate, up = exact_case(m, 300, 136)
    ops = [mxq.bf16_operand(t.bfloat16()) for t in (x, wg, wu)]
    clean, saved = mxq.gemm_gated(*ops, act=act), torch.empty((2, m, 300), device="cuda")
    ops[0].codes[1, 70] = NAN
    y = mxq.gemm_gated(*ops, act=act, saved=saved)
    others = torch.arange(m, device="cuda") != 1
    assert bool(y[1].isnan().all()) and bool(saved[:, 1].isnan().all())
    assert torch.equal(y[others], clean[others]) and bool(saved[:, others].isfinite().all())
