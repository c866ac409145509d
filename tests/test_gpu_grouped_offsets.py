"""Offsets of products grouped by expert that are not sorted: rows counted in
so many groups that the tiles no longer fit 32 signed bits."""
import pytest

from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m", [1 << 22, (1 << 22) + 77])
def test_rows_counted_in_many_groups(m):
    """Every other one of 65536 groups claims all rows: 2**31 tiles of 64 rows
    and more.  Nothing outside the output is written, and as all experts have the
    same weights here the rows hold their product whichever group took them."""
    import torch
    import fp8_quantized_linear_mxq_amd as mxq
    gu.say(f"grouped int8, {m} rows in every other of 65536 groups")
    groups, n, k = 65536, 128, 32
    g = torch.Generator(device="cuda")
    g.manual_seed(m)
    codes = lambda r: torch.randint(-3, 4, (r, k), generator=g, device="cuda").to(torch.int8)
    a, one = codes(m), codes(n)
    w = one.repeat(groups, 1)
    off = torch.zeros(groups + 1, dtype=torch.int32, device="cuda")
    off[1::2] = m
    guard = torch.full((m + 128, n), -7.5, dtype=torch.bfloat16, device="cuda")
    mxq.gemm_grouped(mxq.int8_operand(a, torch.ones(m, device="cuda")),
                     mxq.int8_operand(w, torch.ones(groups * n, device="cuda")), off, out=guard[64:64 + m])
    assert bool((guard[:64] == -7.5).all()) and bool((guard[64 + m:] == -7.5).all())
    for r in range(0, m, 1 << 19):
        want = a[r:r + (1 << 19)].float() @ one.float().t().contiguous()
        assert torch.equal(guard[64:64 + m][r:r + (1 << 19)], want.bfloat16())
