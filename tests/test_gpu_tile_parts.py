"""Products in two launches, whole rounds of the largest tiles and the rest in
another shape: exact sums over outputs whose cut falls on columns or on rows,
and rests with K split."""
import pytest
import torch

import fp8_quantized_linear_mxq_amd as mxq
from tests import gpu_util as gu
from tests.test_gpu_fp8 import bf16, gen, whole
from tests.test_gpu_gated import exact_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n,k", [(4400, 4401, 4096), (8300, 2200, 4128)])
def test_fp8(m, n, k):
    gu.say(f"fp8 {m}x{n}x{k}, exact sums")
    g = gen(m + n)
    (a, av), (w, wv) = whole(g, m, k, False, density=0.1), whole(g, n, k, True, density=0.1)
    assert torch.equal(mxq.gemm(a, w), bf16(av @ wv.t()))
    perm = torch.randperm(n + 3, generator=g, device="cuda")[:n].int()
    bias = torch.randint(-4, 5, (n + 3,), generator=g, device="cuda").bfloat16()
    out = torch.full((m, n + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    mxq.gemm_mixed(a, [w], perm, n + 3, bias=bias, out=out)
    want = torch.full((m, n + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    want[:, perm.long()] = bf16(av @ wv.t() + bias.double()[perm.long()])
    assert torch.equal(out, want)


@pytest.mark.parametrize("m,n,k", [(4400, 2200, 4096), (8300, 1101, 4128), (33000, 200, 4096)])
def test_gated_fp8(m, n, k):
    gu.say(f"gated fp8 {m}x{n}x{k}, exact sums")
    g = gen(m + n)
    d = min(1.0, 80 / k)
    (a, av), (wg, gv), (wu, uv) = whole(g, m, k, False, -1, 2, d), whole(g, n, k, True, -1, 2, d), whole(g, n, k, True, -1, 2, d)
    for q, v, first in ((a, av, 32.0), (wg, gv, 64.0), (wu, uv, 0.0)):
        q.codes.view(torch.float8_e4m3fn)[:, 0] = torch.tensor(first, device="cuda").to(torch.float8_e4m3fn)
        s = (q.scales[0] if q is a else q.scales[:, 0].repeat_interleave(128)[:n]).double()
        v[:, 0] = first * s
    gate, up = av @ gv.t(), av @ uv.t()
    assert float(gate.min()) >= 64 and float((gate * up).abs().max()) < 2 ** 24 / 16
    assert torch.equal(mxq.gemm_gated(a, wg, wu), bf16(gate * up))


# forward by columns and rows; gradients by columns and rows, with and without a split K
@pytest.mark.parametrize("m,n,k", [(8300, 2200, 2056), (17000, 1100, 2056), (33000, 200, 520), (8300, 600, 4104),
                                   (8300, 1100, 2056), (2300, 4400, 4104), (4400, 2200, 4104), (8192, 5632, 2048)])
def test_gated(m, n, k):
    gu.say(f"gated {m}x{n}x{k} bf16, exact sums")
    x, wg, wu, dy, gate, up = exact_case(m, n, k)
    ops = [mxq.bf16_operand(t.bfloat16()) for t in (x, wg, wu)]
    saved = torch.empty((2, m, n), device="cuda")
    want = bf16(gate * up)
    assert torch.equal(mxq.gemm_gated(*ops), want)
    assert torch.equal(mxq.gemm_gated(*ops, saved=saved), want)
    assert torch.equal(saved.double(), torch.stack([gate, up]))
    got = mxq.gemm_gated_backward(dy.bfloat16(), *ops, saved)
    dg, du = dy.double() * up, dy.double() * gate
    for a, b in zip(got, (dg @ wg.double() + du @ wu.double(), dg.t() @ x.double(), du.t() @ x.double())):
        assert torch.equal(a, bf16(b))
