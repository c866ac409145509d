"""Calls given a stream: outputs and workspaces are allocated on it, so that
their memory is not handed to other work before the kernels there are done."""
import pytest
import torch

import fp8_quantized_linear_mxq_amd as mxq

pytestmark = pytest.mark.gpu


def _weights(n, k, fmt):
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    return mxq.quantize(torch.randn(n, k, generator=g, device="cuda"), fmt)


def _calls():
    x, m, n, k = torch.ones(8, 256, device="cuda"), 8, 64, 256
    x16 = x.bfloat16()
    perm = torch.arange(n, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 3, m], dtype=torch.int32, device="cuda")
    i8 = mxq.quantize(x, mxq.INT8), _weights(n, k, mxq.INT8)
    m4 = mxq.quantize(x, mxq.MXFP4), _weights(n, k, mxq.INT4)
    img, wc = mxq.quantize(torch.ones(16, 128, device="cuda"), mxq.MXFP8), _weights(n, 9 * 128, mxq.INT4)
    w, l1 = torch.ones(n, k, device="cuda"), torch.ones(16, k, dtype=torch.bfloat16, device="cuda")
    return {
        "quantize": lambda s: mxq.quantize(x, mxq.NVFP4, stream=s),
        "gemm": lambda s: mxq.gemm(*i8, stream=s),
        "gemm int4": lambda s: mxq.gemm(*m4, stream=s),
        "gemm_grouped": lambda s: mxq.gemm_grouped(*i8, off, stream=s),
        "gemm_mixed": lambda s: mxq.gemm_mixed(i8[0], [i8[1]], perm, n, stream=s),
        "gemm_mixed int4": lambda s: mxq.gemm_mixed(m4[0], [m4[1]], perm, n, stream=s),
        "conv": lambda s: mxq.conv3x3_gemm_mixed(img, 4, 4, [wc], perm, n, stream=s),
        "qk_norm_rope": lambda s: mxq.qk_norm_rope(x16, 2, 1, 64, stream=s),
        "pack_l1t": lambda s: mxq.pack_l1t(l1, stream=s),
        "select_format": lambda s: mxq.select_format(w, stream=s),
        "quantize_mse": lambda s: mxq.quantize_mse(w, mxq.MXFP4, stream=s),
        "lowrank_split": lambda s: mxq.lowrank_split(w, 8, stream=s),
    }


@pytest.mark.parametrize("name", ["quantize", "gemm", "gemm int4", "gemm_grouped", "gemm_mixed", "gemm_mixed int4",
                                  "conv", "qk_norm_rope", "pack_l1t", "select_format", "quantize_mse",
                                  "lowrank_split"])
def test_allocations_are_the_given_streams(name):
    """The allocator's record names the stream of every block it hands out."""
    call = _calls()[name]
    want = call(None)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.memory._record_memory_history(context=None, max_entries=10000)
    try:
        got = call(s)
        trace = torch.cuda.memory._snapshot()["device_traces"][torch.cuda.current_device()]
    finally:
        torch.cuda.memory._record_memory_history(enabled=None)
    made = [e for e in trace if e["action"] == "alloc"]
    assert made and all(e["stream"] == s.cuda_stream for e in made)
    s.synchronize()

    def same(a, b):
        if isinstance(a, mxq.QTensor):
            return torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
        if isinstance(a, tuple):
            return all(same(p, q) for p, q in zip(a, b))
        return torch.equal(a, b)

    if name != "quantize":   # its padding columns are never written
        assert same(got, want)
