"""Which kernel a product runs on, and that kernel's main loop, for the int8
products and those grouped by expert: each case names the kernel that it was
written for (read from a trace of the call), so a threshold that moves cannot
take it to another one unnoticed.  Results against float64 products on the
device, within the bound of every route."""
import re

import pytest
import torch

import fp8_quantized_linear_mxq_amd as mxq
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


def traced(call):
    """(result, names of the library's kernels) of one call."""
    from torch.profiler import ProfilerActivity, profile
    torch.cuda.synchronize()
    with profile(activities=[ProfilerActivity.CUDA], acc_events=True) as p:
        y = call()
        torch.cuda.synchronize()
    return y, [m.group(1) for m in (re.search(r"mxq::.*?(\w+<[^>]*>)\(", e.name) for e in p.events()) if m]


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def operand(g, pair, rows, k, act=False):
    """(operand, exact float64 values)"""
    if pair == "BF16" and act:
        x = torch.randn(rows, k, generator=g, device="cuda").bfloat16()
        return mxq.bf16_operand(x), x.double()
    if pair == "INT8":
        q = (40 * torch.randn(rows, k, generator=g, device="cuda")).round().clamp(-127, 127).to(torch.int8)
        s = torch.exp(4 * torch.rand(rows, generator=g, device="cuda") - 4)
        return mxq.int8_operand(q, s), q.double() * s.double()[:, None]
    codes = torch.randint(0, 256, (rows, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(118, 132, (rows, k // 32), generator=g, device="cuda", dtype=torch.uint8)
    table = torch.tensor(_E2M1 + [-v for v in _E2M1], dtype=torch.float64, device="cuda")
    v = torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], dim=2).view(rows, -1, 32)
    return mxq.QTensor(mxq.MXFP4, rows, k, codes, scales), (v * torch.exp2(scales.double() - 127)[:, :, None]).view(rows, -1)


def within(y, av, wv, bias=None, extra=None, extra_s=None):
    """The bound of every route, for float64 operands on the device."""
    wt = wv.t().contiguous()
    want, s = av @ wt, av.abs() @ wt.abs()
    if bias is not None:
        want = want + bias.double()
    if extra is not None:
        want, s = want + extra, s + extra_s
    err, tol = (y.double() - want).abs(), 1e-5 * (1 + 2.0 ** -8) * s + 2.0 ** -8 * want.abs() + 2.0 ** -133
    assert bool((err <= tol).all()), f"worst {float((err / tol).max()):.3g} of the bound"


# ---- int8 x int8 ------------------------------------------------------------

RING = "gemm_i8_ring_kernel<%d, %s, %s, %s>"
# tiles of 64, 128 and 256, and the staged 64: a size of each, ragged
TILES = {(1, "false"): (1530, 1400), (2, "false"): (2290, 3990), (4, "false"): (4090, 4080), (1, "true"): (500, 1010)}
# K-tiles of 128: one to three turns of the five-K-tile loop with every number
# left over, and with and without a partial last one
LOOP_K = [640, 672, 768, 1152, 1184, 1280, 1440, 1536, 1664, 1792, 1920, 2080]


@pytest.mark.parametrize("k", LOOP_K)
@pytest.mark.parametrize("tile", TILES)
def test_int8_main_loop(tile, k):
    m, n = TILES[tile]
    gu.say(f"int8 {m}x{n}x{k}, tiles {tile}")
    g = generator(k)
    (a, av), (w, wv) = operand(g, "INT8", m, k), operand(g, "INT8", n, k)
    bias = torch.randn(n, generator=g, device="cuda").bfloat16()
    y, ran = traced(lambda: mxq.gemm(a, w, bias=bias))
    assert ran == [RING % (tile[0], "false", "false", tile[1])]
    within(y, av, wv, bias)


@pytest.mark.parametrize("k", [96, 1184, 1920])
@pytest.mark.parametrize("tile", [t for t in TILES if t[0] < 4])
def test_int8_lowrank_column_map(tile, k):
    """The low-rank branch and a column map on each tile that takes them."""
    m, n = TILES[tile]
    r, n_out = 32, n + 13
    gu.say(f"int8 {m}x{n}x{k} with low rank and map, tiles {tile}")
    g = generator(k + 1)
    (a, av), (w, wv) = operand(g, "INT8", m, k), operand(g, "INT8", n, k)
    u = 4 * torch.randn(m, r, generator=g, device="cuda")
    l2 = torch.randn(n_out, r, generator=g, device="cuda").bfloat16()
    cols = torch.randperm(n_out, generator=g, device="cuda")[:n].int()
    out = torch.full((m, n_out), -7.0, dtype=torch.bfloat16, device="cuda")
    y, ran = traced(lambda: mxq.gemm(a, w, n_out=n_out, w_out_col=cols, u=u, l2t=l2, out=out))
    assert ran == [RING % (tile[0], "true", "false", tile[1])]
    ud, ld = u.double(), l2[cols.long()].double().t().contiguous()
    within(y[:, cols.long()], av, wv, extra=ud @ ld, extra_s=ud.abs() @ ld.abs())
    rest = torch.ones(n_out, dtype=torch.bool, device="cuda")
    rest[cols.long()] = False
    assert bool((y[:, rest] == -7).all())


@pytest.mark.parametrize("tile", TILES)
def test_int8_longest_sum(tile):
    """K = 2**17 with the largest codes: the sum only just stays within int32."""
    m, n = TILES[tile]
    k = 1 << 17
    gu.say(f"int8 {m}x{n}x{k}, tiles {tile}")
    a = torch.full((m, k), 127, dtype=torch.int8, device="cuda")
    w = torch.full((n, k), 127, dtype=torch.int8, device="cuda")
    w[7] = -127
    a[5] = -127
    one = lambda r: torch.ones(r, device="cuda")
    y, ran = traced(lambda: mxq.gemm(mxq.int8_operand(a, one(m)), mxq.int8_operand(w, one(n))))
    # the fp32 of a whole K may make another tile the faster one
    assert len(ran) == 1 and ran[0].startswith("gemm_i8_ring_kernel")
    want = torch.full((m, n), 127.0 * 127 * k, device="cuda").bfloat16()
    want[5] = -want[5]
    want[:, 7] = -want[:, 7]
    assert torch.equal(y, want)


# ---- products grouped by expert ---------------------------------------------

MXK = "gemm_mx_kernel<%d, %d, %d, %s, false, %s, true>"
DQP = "grouped_dqp_kernel<3, 2, %d, %d, %d, %s, %d>"
FEW = "gemm_few_kernel<%d, %d, true>"


def spread(rows, groups, seed):
    """Uneven sizes, some of them zero, that add up to `rows`."""
    g = torch.Generator().manual_seed(seed)
    p = torch.rand(groups, generator=g) ** 3
    p[::5] = 0
    n = (p / p.sum() * rows).floor().int()
    n[groups // 2] += rows - int(n.sum())
    return n.tolist()


def offsets(sizes, first=0):
    return (torch.tensor([0] + sizes).cumsum(0) + first).int().cuda()


# (pair, sizes, N, K, kernel)
GROUPED = [
    ("INT8", spread(1300, 90, 1), 700, 1184, RING % (1, "false", "true", "false")),
    ("INT8", spread(3000, 8, 2), 1500, 1312, RING % (2, "false", "true", "false")),
    ("INT8", spread(16000, 8, 3), 2000, 1440, RING % (2, "false", "true", "false")),
    ("INT8", spread(15000, 4, 3), 2000, 1440, RING % (4, "false", "true", "false")),
    ("INT8", spread(900, 6, 4), 500, 1184, RING % (1, "false", "true", "true")),
    ("INT8", spread(150, 70, 5), 210, 4640, FEW % (0, 1)),
    ("INT8", spread(130, 4, 5), 620, 1184, FEW % (0, 2)),
    # few rows per group, few tiles
    ("MXFP4", spread(600, 70, 6), 1000, 512, MXK % (1, 1, 2, "false", "true")),
    ("MXFP4", spread(600, 70, 6), 1000, 640, MXK % (1, 1, 2, "false", "false")),
    ("MXFP4", spread(500, 70, 7), 300, 4608, MXK % (1, 1, 2, "true", "true")),
    ("MXFP4", spread(1500, 6, 7), 300, 4224, MXK % (1, 1, 2, "true", "false")),
    ("MXFP4", spread(4100, 70, 8), 900, 512, MXK % (2, 2, 2, "false", "true")),
    ("MXFP4", spread(4100, 6, 8), 1000, 896, MXK % (2, 2, 2, "false", "false")),
    ("MXFP4", spread(4100, 70, 9), 600, 4608, MXK % (2, 2, 2, "true", "true")),
    ("MXFP4", spread(4100, 6, 9), 1000, 4224, MXK % (2, 2, 2, "true", "false")),
    ("MXFP4", spread(13900, 4, 10), 3000, 1024, MXK % (2, 4, 4, "false", "true")),
    ("MXFP4", spread(13900, 4, 10), 3000, 384, MXK % (2, 4, 4, "false", "false")),
    ("MXFP4", spread(15800, 4, 11), 1700, 1024, MXK % (2, 3, 4, "false", "true")),
    ("MXFP4", spread(15800, 4, 11), 1700, 384, MXK % (2, 3, 4, "false", "false")),
    ("MXFP4", [1, 0, 0, 3, 1], 70, 8320, FEW % (1, 2)),
    # the decode batch: 32-row tiles, wide where those fill the GPU
    ("BF16", spread(64, 32, 12), 2048, 1152, DQP % (1, 2, 1, "false", 4)),
    ("BF16", spread(700, 70, 12), 700, 384, DQP % (1, 2, 1, "false", 4)),
    ("BF16", spread(1000, 31, 13), 400, 512, DQP % (1, 1, 1, "false", 4)),
    ("BF16", spread(300, 40, 13), 500, 1280, DQP % (1, 1, 1, "false", 4)),
    ("BF16", spread(1000, 31, 14), 400, 4224, DQP % (1, 1, 1, "true", 4)),
    ("BF16", spread(70, 70, 14), 300, 4992, FEW % (2, 2)),
    ("BF16", spread(80, 80, 14), 400, 4992, DQP % (1, 1, 1, "true", 4)),
    ("BF16", spread(4100, 70, 15), 400, 640, DQP % (2, 1, 1, "false", 4)),
    ("BF16", spread(7000, 70, 15), 2000, 640, DQP % (2, 2, 1, "false", 4)),
    ("BF16", spread(4100, 70, 16), 400, 4224, DQP % (2, 2, 2, "true", 2)),
    ("BF16", [0, 2, 1, 0, 4], 70, 8320, FEW % (2, 2)),
]


@pytest.mark.parametrize("case", range(len(GROUPED)))
def test_grouped_kernel(case):
    pair, sizes, n, k, kernel = GROUPED[case]
    e, m = len(sizes), sum(sizes)
    gu.say(f"grouped {pair} E={e} M={m} N={n} K={k}: {kernel}")
    g = generator(case)
    (a, av), (w, wv) = operand(g, pair, m, k, act=True), operand(g, pair, e * n, k)
    bias = torch.randn(e, n, generator=g, device="cuda").bfloat16()
    y, ran = traced(lambda: mxq.gemm_grouped(a, w, offsets(sizes), bias=bias))
    assert ran == [kernel]
    lo = 0
    for i, s in enumerate(sizes):
        if s:
            within(y[lo:lo + s], av[lo:lo + s], wv[i * n:(i + 1) * n], bias[i])
        lo += s


# Tiled sizes (64- and 128-row tiles or larger) for what the offsets can hold
TILED = [("INT8", 1500, 900, 288), ("INT8", 9000, 2100, 288), ("MXFP4", 1500, 300, 384), ("MXFP4", 9000, 1100, 384),
         ("MXFP4", 14000, 3000, 128), ("BF16", 1500, 300, 384), ("BF16", 9000, 2100, 128)]


def tiled(case, seed):
    pair, m, n, k = TILED[case]
    g = generator(seed)
    (a, av), (w, wv) = operand(g, pair, m, k, act=True), operand(g, pair, 4 * n, k)
    guard = torch.full((m + 128, n), -7.0, dtype=torch.bfloat16, device="cuda")

    def run(off):
        off = torch.tensor(off, dtype=torch.int32, device="cuda")
        _, ran = traced(lambda: mxq.gemm_grouped(a, w, off, out=guard[64:64 + m]))
        assert len(ran) == 1 and not ran[0].startswith("gemm_few")
        assert bool((guard[:64] == -7).all()) and bool((guard[64 + m:] == -7).all())
        return guard[64:64 + m]

    def check(y, group, lo, hi):
        within(y[lo:hi], av[lo:hi], wv[group * n:(group + 1) * n])
    return m, run, check


@pytest.mark.parametrize("case", range(len(TILED)))
def test_tiled_rows_outside_all_groups(case):
    m, run, check = tiled(case, 20)
    y = run([37, 300, 300, m - 450, m - 91])
    check(y, 0, 37, 300), check(y, 2, 300, m - 450), check(y, 3, m - 450, m - 91)
    assert bool((y[:37] == -7).all()) and bool((y[m - 91:] == -7).all())


@pytest.mark.parametrize("case", range(len(TILED)))
def test_tiled_no_rows_in_any_group(case):
    m, run, _ = tiled(case, 21)
    for at in (0, 100, m):
        assert bool((run([at] * 5) == -7).all())


@pytest.mark.parametrize("case", range(len(TILED)))
def test_tiled_offsets_out_of_range(case):
    """Values outside [0, M] are clamped; after decreasing ones rows are
    unspecified, and nothing outside the output is written."""
    m, run, check = tiled(case, 22)
    y = run([-50, 260, 700, 700, m + 10000])
    check(y, 0, 0, 260), check(y, 1, 260, 700), check(y, 3, 700, m)
    run([m - 200, 30, 2 ** 31 - 1, -2 ** 31, m - 7])
    run([0, m, 0, m, 0])
    run([-1, -2 ** 31, 2 ** 31 - 1, 5, m])


@pytest.mark.parametrize("case", range(len(TILED)))
def test_tiled_in_a_graph_with_new_offsets(case):
    pair, m, n, k = TILED[case]
    g = generator(23)
    (a, _), (w, _) = operand(g, pair, m, k, act=True), operand(g, pair, 4 * n, k)
    off = torch.tensor([0, m, m, m, m], dtype=torch.int32, device="cuda")
    out = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    mxq.gemm_grouped(a, w, off, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mxq.gemm_grouped(a, w, off, out=out)
    for i in range(4):
        cut = torch.randint(0, m + 1, (3,), generator=torch.Generator().manual_seed(i)).sort().values.tolist()
        off.copy_(torch.tensor([0] + cut + [m], dtype=torch.int32))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, mxq.gemm_grouped(a, w, off))


@pytest.mark.parametrize("m,n", [(700, 900), (4090, 4080)])
def test_one_group_is_the_plain_product(m, n):
    """On the staged tiles and on larger ones."""
    g = generator(24)
    (a, _), (w, _) = operand(g, "INT8", m, 1184), operand(g, "INT8", n, 1184)
    off = torch.tensor([0, m], dtype=torch.int32, device="cuda")
    y, ran = traced(lambda: mxq.gemm_grouped(a, w, off))
    assert len(ran) == 1 and ran[0].startswith("gemm_i8_ring_kernel")
    assert torch.equal(y, mxq.gemm(a, w))


@pytest.mark.parametrize("k", [32, 96, 160, 672, 2080])
def test_grouped_int8_partial_k(k):
    sizes, n = [900, 0, 1300, 1, 700], 900
    g = generator(k)
    (a, av), (w, wv) = operand(g, "INT8", sum(sizes), k), operand(g, "INT8", len(sizes) * n, k)
    y, ran = traced(lambda: mxq.gemm_grouped(a, w, offsets(sizes)))
    assert len(ran) == 1 and ran[0].startswith("gemm_i8_ring_kernel")
    lo = 0
    for i, s in enumerate(sizes):
        if s:
            within(y[lo:lo + s], av[lo:lo + s], wv[i * n:(i + 1) * n])
        lo += s
