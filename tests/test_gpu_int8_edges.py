"""int8 quantize outside its contract: what it writes stays codes."""
import pytest
import torch

import fp8_quantized_linear_mxq_amd as mxq
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("had", [0, 16])
@pytest.mark.parametrize("k", [256, 4096])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_nan_and_infinity_give_valid_codes(dtype, k, had):
    """NaNs of any payload and sign, infinities: every code lies in [-127, 127],
    and rows without them are what they are alone."""
    gu.say(f"int8 quantize of NaN and Inf, {dtype}, K={k}, rotation {had}")
    g = torch.Generator(device="cuda")
    g.manual_seed(k)
    x = torch.randn(600, k, generator=g, device="cuda").to(dtype)
    clean = x.clone()
    low = torch.arange(256, device="cuda")
    if dtype == torch.float32:
        bits = torch.cat([0x7FC00000 | low, 0x7F800100 | low, (0x7FC00000 | low) - (1 << 31)]).int()
    else:
        bits = torch.cat([0x7F80 | (low & 127), (0x7F80 | (low & 127)) - (1 << 15)]).short()
    bits = bits[:590]
    x.view(bits.dtype)[torch.arange(len(bits), device="cuda"), torch.arange(len(bits), device="cuda") % k] = bits
    x[590, 3], x[591] = float("inf"), float("-inf")
    q = mxq.quantize(x, mxq.INT8, hadamard=had).codes.view(torch.int8)
    assert int(q.min()) >= -127
    want = mxq.quantize(clean, mxq.INT8, hadamard=had).codes.view(torch.int8)
    assert torch.equal(q[592:], want[592:])
