"""The torch binding of quantize, gemm, gemm_grouped and qk_norm_rope: tensors
that the C ABI could not tell from right ones are refused before the call,
and strides that do not matter are accepted."""
import pytest
import torch

import fp8_quantized_linear_mxq_amd as mxq

pytestmark = pytest.mark.gpu


def operands(m=4, n=32, k=64):
    codes = lambda r: torch.arange(r * k, device="cuda").remainder(5).sub(2).to(torch.int8).view(r, k)
    return (mxq.int8_operand(codes(m), torch.ones(m, device="cuda")),
            mxq.int8_operand(codes(n), torch.ones(n, device="cuda")))


@pytest.mark.parametrize("x", [
    lambda: torch.zeros(4, 64),                                                  # host memory
    lambda: torch.zeros(4, 64, dtype=torch.float16, device="cuda"),
    lambda: torch.zeros(4, 64, dtype=torch.int32, device="cuda"),
    lambda: torch.zeros(4, 128, device="cuda")[:, ::2],
    lambda: torch.zeros(64, 4, device="cuda").t(),
], ids=["host", "float16", "int32", "column stride", "transposed"])
@pytest.mark.parametrize("fmt", [mxq.INT8, mxq.MXFP4])
def test_quantize_refuses(x, fmt):
    with pytest.raises(ValueError):
        mxq.quantize(x(), fmt)


def test_quantize_out_has_the_rows():
    out = mxq.quantize(torch.ones(2, 64, device="cuda"), mxq.INT8)
    out.rows = 4
    with pytest.raises(ValueError):
        mxq.quantize(torch.ones(4, 64, device="cuda"), mxq.INT8, out=out)


def test_one_row_of_any_stride():
    a, w = operands()
    x = torch.linspace(-1, 1, 64, device="cuda").view(64, 1).t()   # [1, 64], row stride 1
    q, want = mxq.quantize(x, mxq.INT8), mxq.quantize(x.clone(memory_format=torch.contiguous_format), mxq.INT8)
    assert torch.equal(q.codes, want.codes) and torch.equal(q.scales, want.scales)
    out = torch.empty(32, 1, dtype=torch.bfloat16, device="cuda").t()
    assert torch.equal(mxq.gemm(q, w, out=out), mxq.gemm(want, w))


BAD_OUT = [
    lambda m, n: torch.empty(m, n, device="cuda"),                                          # float32
    lambda m, n: torch.empty(m - 1, n, dtype=torch.bfloat16, device="cuda"),
    lambda m, n: torch.empty(m, n - 1, dtype=torch.bfloat16, device="cuda"),
    lambda m, n: torch.empty(n, m, dtype=torch.bfloat16, device="cuda").t(),
    lambda m, n: torch.empty(m, n, dtype=torch.bfloat16),                                   # host memory
]


@pytest.mark.parametrize("out", BAD_OUT)
def test_product_refuses_out(out):
    a, w = operands()
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        mxq.gemm(a, w, out=out(4, 32))
    with pytest.raises(ValueError):
        mxq.gemm_grouped(a, w, off, out=out(4, 32))


@pytest.mark.parametrize("bias", [lambda: torch.zeros(32, device="cuda"),
                                  lambda: torch.zeros(31, dtype=torch.bfloat16, device="cuda"),
                                  lambda: torch.zeros(64, dtype=torch.bfloat16, device="cuda")[::2]])
def test_product_refuses_bias(bias):
    a, w = operands()
    with pytest.raises(ValueError):
        mxq.gemm(a, w, bias=bias())
    with pytest.raises(ValueError):
        mxq.gemm_grouped(a, w, torch.tensor([0, 4], dtype=torch.int32, device="cuda"), bias=bias())


@pytest.mark.parametrize("off", [lambda: torch.tensor([0, 4], device="cuda"),
                                 lambda: torch.tensor([0, 4], dtype=torch.int32),
                                 lambda: torch.tensor([0, 1, 4, 9], dtype=torch.int32, device="cuda")[::2]])
def test_grouped_refuses_offsets(off):
    a, w = operands()
    with pytest.raises(ValueError):
        mxq.gemm_grouped(a, w, off())


def test_operand_of_host_memory():
    a, w = operands()
    with pytest.raises(ValueError):
        mxq.gemm(mxq.int8_operand(a.codes.cpu(), a.scales.cpu()), w)
    with pytest.raises(ValueError):
        mxq.gemm(a, mxq.int8_operand(w.codes, w.scales.cpu()))


def test_given_stream_owns_what_it_writes():
    a, w = operands()
    want = mxq.gemm(a, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [mxq.gemm(a, w, stream=s) for _ in range(4)]
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    outs.append(mxq.gemm_grouped(a, w, off, stream=s))
    torch.cuda.current_stream().wait_stream(s)
    for o in outs:
        assert torch.equal(o, want)
