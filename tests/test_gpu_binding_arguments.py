"""Arguments of the torch binding that the C ABI sees as bare addresses: the
wrong type or size is refused before the call, what can be read is taken."""
import pytest
import torch

import fp8_quantized_linear_mxq_amd as mxq

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def zeros(*size, dtype=F32, device="cuda"):
    return torch.zeros(size, dtype=dtype, device=device)


# ---- quantize: L1, u, the static tensor scale ------------------------------

M, K, R = 6, 256, 32


@pytest.mark.parametrize("u", [
    lambda: zeros(M - 1, R), lambda: zeros(M, R - 1), lambda: zeros(M, R, dtype=BF16),
    lambda: zeros(M, R, dtype=torch.float64), lambda: zeros(R, M).t(), lambda: zeros(M, 2 * R)[:, ::2],
    lambda: zeros(M * R), lambda: zeros(M, R, device="cpu"),
], ids=["rows", "rank", "bf16", "f64", "transposed", "column stride", "1-D", "host"])
@pytest.mark.parametrize("fmt", [mxq.INT8, mxq.MXFP4])
def test_quantize_refuses_u(u, fmt):
    with pytest.raises(ValueError):
        mxq.quantize(zeros(M, K, dtype=BF16), fmt, l1t=zeros(R, K, dtype=BF16), u=u())


@pytest.mark.parametrize("l1t", [
    lambda: zeros(R, K), lambda: zeros(R, K, dtype=torch.float16), lambda: zeros(R, K - 32, dtype=BF16),
    lambda: zeros(R, K + 32, dtype=BF16), lambda: zeros(R, K + 32, dtype=BF16)[:, :K],
    lambda: zeros(K, R, dtype=BF16).t(), lambda: zeros(R * K, dtype=BF16), lambda: zeros(R, K, dtype=BF16, device="cpu"),
], ids=["f32", "f16", "narrow", "wide", "row stride", "transposed", "1-D", "host"])
@pytest.mark.parametrize("fmt", [mxq.INT8, mxq.MXFP4])
def test_quantize_refuses_l1t(l1t, fmt):
    with pytest.raises(ValueError):
        mxq.quantize(zeros(M, K, dtype=BF16), fmt, l1t=l1t(), u=zeros(M, R))


@pytest.mark.parametrize("g", [lambda: zeros(1, dtype=torch.float64), lambda: zeros(1, dtype=BF16), lambda: zeros(0),
                               lambda: zeros(1, device="cpu")], ids=["f64", "bf16", "empty", "host"])
def test_quantize_refuses_static_scale(g):
    with pytest.raises(ValueError):
        mxq.quantize(zeros(M, K), mxq.NVFP4, static_tensor_scale=g())


def test_quantize_takes_strided_u_and_bits():
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    x = torch.randn(M, K, generator=g, device="cuda").to(BF16)
    l1 = torch.randn(R, K, generator=g, device="cuda").to(BF16)
    u, wide = zeros(M, R), zeros(M + 2, R + 8)
    want = mxq.quantize(x, mxq.INT8, l1t=l1, u=u)
    got = mxq.quantize(x, mxq.INT8, l1t=l1.view(torch.int16), u=wide)
    assert torch.equal(got.codes, want.codes) and torch.equal(wide[:M, :R], u)
    assert not bool(wide[M:].any()) and not bool(wide[:, R:].any())
