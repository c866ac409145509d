"""FP8 operands near the largest numbers of rows and columns: indexes that pass 2**30
and 2**31 in rows, columns and bytes."""
import pytest
import torch

import fp8_quantized_linear_mxq_amd as mxq
from tests import gpu_util as gu
from tests.test_gpu_many_workgroups import memory, room, same_blocks   # noqa: F401 (memory: a fixture of every test)

pytestmark = pytest.mark.gpu

BLOCK = 1 << 20


def rows_of(m, k):
    """(operand of m rows that repeat the same 2**20, that block's float64 values)"""
    g = torch.Generator(device="cuda")
    g.manual_seed(m % 1000)
    v = torch.randint(-3, 4, (BLOCK, k), generator=g, device="cuda").float()
    s = torch.exp2(torch.randint(-3, 4, (BLOCK,), generator=g, device="cuda").float())
    reps = -(-m // BLOCK)
    codes = v.to(torch.float8_e4m3fn).view(torch.uint8).repeat(reps, 1)[:m]
    return mxq.fp8_operand(codes, s.repeat(reps)[None, :m]), v.double() * s.double()[:, None]


def weights(n, k):
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    v = torch.randint(-3, 4, (n, k), generator=g, device="cuda").float()
    return mxq.fp8_operand(v.to(torch.float8_e4m3fn), torch.ones(((n + 127) // 128, 1), device="cuda"), tile=True), v.double()


@pytest.mark.parametrize("m,n", [((1 << 30) + 30, 8), ((1 << 31) - 512, 1)])
def test_products_of_many_rows(m, n):
    """Every row has the scale of its own: the first tile is 2**30 rows and more from the last."""
    room(110)
    gu.say(f"fp8 {m} x {n} x 32")
    (a, av), (w, wv) = rows_of(m, 32), weights(n, 32)
    y = mxq.gemm(a, w)
    want = (av @ wv.t()).float().bfloat16()
    same_blocks(y, want)
    rest = m % BLOCK
    assert torch.equal(y[m - rest:], want[:rest])


def test_products_of_many_columns():
    room(90)
    n = (1 << 31) - 512
    gu.say(f"fp8 1 x {n} x 32")
    (w, wv), (a, av) = rows_of(n, 32), rows_of(1, 32)
    tile = torch.exp2((torch.arange(-(-n // 128), device="cuda") % 8).float())   # BLOCK / 128 is a multiple of 8
    y = mxq.gemm(a, mxq.fp8_operand(w.codes, tile[:, None], tile=True))
    v = w.codes[:BLOCK].view(torch.float8_e4m3fn).double() * tile[:BLOCK // 128].double().repeat_interleave(128)[:, None]
    want = (av[:1] @ v.t()).float().bfloat16()[0]
    same_blocks(y[0], want)
    rest = n % BLOCK
    assert torch.equal(y[0, n - rest:], want[:rest])


@pytest.mark.parametrize("fmt", [mxq.FP8, mxq.FP8_TILE])
def test_quantize_of_wide_rows(fmt):
    """As many columns as an operand can have."""
    room(30)
    cols = (1 << 31) - 32
    gu.say(f"fp8 quantize 1 x {cols}, format {fmt}")
    block = torch.randn((1, BLOCK), device="cuda").bfloat16()
    x = block.repeat(1, 1 << 11)[:, :cols]
    q, want = mxq.quantize(x, fmt), mxq.quantize(block, fmt)
    whole = cols // BLOCK
    same_blocks(q.codes[0, :whole * BLOCK], want.codes[0])
    same_blocks(q.scales.view(-1)[:whole * (BLOCK // 128)], want.scales.view(-1))
    end = mxq.quantize(block[:, :cols % BLOCK], fmt)   # ends inside a K-block
    assert torch.equal(q.codes[0, whole * BLOCK:], end.codes[0])
    assert torch.equal(q.scales.view(-1)[whole * (BLOCK // 128):], end.scales.view(-1))
