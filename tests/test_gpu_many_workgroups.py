"""Inputs whose grids reach 2**32 threads, where a one-dimensional launch is cut
off without an error: tens of millions of tokens, or of output columns."""
import pytest
import torch

import fp8_quantized_linear_mxq_amd as mxq
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

GB = 1 << 30


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def room(gigabytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gigabytes * GB:
        pytest.skip(f"needs {gigabytes} GiB of free device memory")


def same_blocks(t, block):
    """Every whole block of rows of t equals `block` (compared 2**22 rows at a time)."""
    n = len(block)
    per = max(1, (1 << 22) // n)
    for r in range(0, len(t) // n, per):
        got = t[r * n:min(r + per, len(t) // n) * n]
        assert bool((got.view(-1, *block.shape) == block).all()), f"rows from {r * n}"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize(dtype):
    room(24)
    gu.say(f"int8 quantize of 70 million rows, {dtype}")
    block = torch.randn(1000, 32, device="cuda").to(dtype)
    x = block.repeat(70_000, 1)
    q, want = mxq.quantize(x, mxq.INT8), mxq.quantize(block, mxq.INT8)
    same_blocks(q.codes, want.codes)
    same_blocks(q.scales, want.scales)


def test_head_norms():
    room(16)
    gu.say("head norms of 70 million tokens")
    block = torch.randn(1000, 8, device="cuda").bfloat16()
    q, _ = mxq.qk_norm_rope(block.repeat(70_000, 1), 1, 0, 8)
    want, _ = mxq.qk_norm_rope(block, 1, 0, 8)
    same_blocks(q, want)


def test_int8_one_token_of_many_columns():
    """Few rows: 16 columns to a workgroup."""
    room(24)
    n, k = 300_000_000, 32
    gu.say(f"int8 1 x {n} x {k}")
    a = torch.randint(-9, 10, (1, k), device="cuda").to(torch.int8)
    w = torch.randint(-9, 10, (1000, k), device="cuda").to(torch.int8)
    y = mxq.gemm(mxq.int8_operand(a, torch.ones(1, device="cuda")),
                 mxq.int8_operand(w.repeat(n // 1000, 1), torch.ones(n, device="cuda")))
    want = (a.float() @ w.float().t().contiguous()).bfloat16()
    same_blocks(y[0], want[0])


def test_int8_many_rows():
    """64-row tiles: 2**24 and more."""
    room(120)
    m, n, k = 1_080_000_000, 8, 32
    gu.say(f"int8 {m} x {n} x {k}")
    a = torch.randint(-9, 10, (1_000_000, k), device="cuda").to(torch.int8)
    w = torch.randint(-9, 10, (n, k), device="cuda").to(torch.int8)
    y = mxq.gemm(mxq.int8_operand(a.repeat(m // 1_000_000, 1), torch.ones(m, device="cuda")),
                 mxq.int8_operand(w, torch.ones(n, device="cuda")))
    same_blocks(y, (a.float() @ w.float().t().contiguous()).bfloat16())


@pytest.mark.parametrize("pair", ["INT8", "MXFP4"])
def test_grouped_many_experts(pair):
    """One row for each of 4096 experts with many columns: 16 x 16 tiles (int8),
    64 x 64 tiles (MXFP4).  Experts of four kinds, told apart by their scales."""
    groups, n, k = (4096, 73_800, 32) if pair == "INT8" else (4096, 264_000, 128)
    room(40 if pair == "INT8" else 120)
    gu.say(f"grouped {pair}, {groups} rows and experts, {n} columns")
    kind = torch.arange(groups, device="cuda") % 4
    off = torch.arange(groups + 1, dtype=torch.int32, device="cuda")
    if pair == "INT8":
        a = mxq.int8_operand(torch.ones(groups, k, dtype=torch.int8, device="cuda"), torch.ones(groups, device="cuda"))
        w = mxq.int8_operand(torch.ones(groups * n, k, dtype=torch.int8, device="cuda"),
                             torch.exp2(kind.float()).repeat_interleave(n))
    else:
        a = mxq.quantize(torch.ones(groups, k, device="cuda"), mxq.MXFP4)
        scales = (127 + kind).to(torch.uint8).repeat_interleave(n)[:, None].repeat(1, 4)
        w = mxq.QTensor(mxq.MXFP4, groups * n, k, torch.full((groups * n, k // 2), 0x22, dtype=torch.uint8, device="cuda"),
                        scales)
    y = mxq.gemm_grouped(a, w, off)
    want = (k * torch.exp2(kind.float())).bfloat16()[:, None]
    for r in range(0, groups, 512):
        assert bool((y[r:r + 512] == want[r:r + 512]).all()), f"rows from {r}"


def test_quantize_lowrank():
    """The projection of 270 million rows, 16 to a workgroup, next to the codes."""
    room(100)
    n = 270_000_000
    gu.say(f"int8 quantize of {n} rows with a rank-16 projection")
    block = torch.randn(1_000_000, 32, device="cuda").bfloat16()
    l1t = torch.randn(16, 32, device="cuda").bfloat16()
    u, want_u = torch.empty(n, 16, device="cuda"), torch.empty(len(block), 16, device="cuda")
    want = mxq.quantize(block, mxq.INT8, l1t=l1t, u=want_u)
    q = mxq.quantize(block.repeat(n // len(block), 1), mxq.INT8, l1t=l1t, u=u)
    same_blocks(u, want_u)
    same_blocks(q.codes, want.codes)
