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


# ---- gemm: column map, low-rank operands -----------------------------------

N = 48


def product(fmt=mxq.INT8, m=M, n=N, k=K):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    return (mxq.quantize(torch.randn(m, k, generator=g, device="cuda"), fmt),
            mxq.quantize(torch.randn(n, k, generator=g, device="cuda"), fmt))


@pytest.mark.parametrize("cols", [
    lambda: torch.randperm(N, device="cuda"), lambda: torch.arange(N - 1, dtype=torch.int32, device="cuda"),
    lambda: torch.arange(2 * N, dtype=torch.int32, device="cuda")[::2], lambda: zeros(N),
    lambda: torch.arange(N, dtype=torch.int32),
], ids=["int64", "short", "strided", "f32", "host"])
@pytest.mark.parametrize("fmt", [mxq.INT8, mxq.MXFP4])
def test_gemm_refuses_column_map(cols, fmt):
    a, w = product(fmt)
    with pytest.raises(ValueError):
        mxq.gemm(a, w, w_out_col=cols())


@pytest.mark.parametrize("u,l2t", [
    (lambda: zeros(M - 1, R), lambda: zeros(N, R, dtype=BF16)), (lambda: zeros(M, R - 16), lambda: zeros(N, R, dtype=BF16)),
    (lambda: zeros(M, R, dtype=BF16), lambda: zeros(N, R, dtype=BF16)), (lambda: zeros(R, M).t(), lambda: zeros(N, R, dtype=BF16)),
    (lambda: zeros(M, R), lambda: zeros(N - 1, R, dtype=BF16)), (lambda: zeros(M, R), lambda: zeros(N, R)),
    (lambda: zeros(M, R), lambda: zeros(N, R, dtype=torch.float16)), (lambda: zeros(M, R), lambda: zeros(R, N, dtype=BF16).t()),
    (lambda: zeros(M, R), lambda: zeros(N, 2 * R, dtype=BF16)[:, :R]), (lambda: zeros(M, R), lambda: zeros(N * R, dtype=BF16)),
], ids=["u rows", "u rank", "u bf16", "u transposed", "l2t rows", "l2t f32", "l2t f16", "l2t transposed",
        "l2t row stride", "l2t 1-D"])
@pytest.mark.parametrize("fmt", [mxq.INT8, mxq.MXFP4])
def test_gemm_refuses_lowrank(u, l2t, fmt):
    a, w = product(fmt)
    with pytest.raises(ValueError):
        mxq.gemm(a, w, u=u(), l2t=l2t())


@pytest.mark.parametrize("fmt", [mxq.INT8, mxq.MXFP4])
def test_gemm_takes_longer_maps_and_strided_u(fmt):
    a, w = product(fmt)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    u, l2t = torch.randn(M, R, generator=g, device="cuda"), torch.randn(N, R, generator=g, device="cuda").to(BF16)
    want = mxq.gemm(a, w, u=u, l2t=l2t)
    wide = zeros(M + 1, R + 4)
    wide[:M, :R] = u
    rev = torch.arange(N, dtype=torch.int32, device="cuda").flip(0)
    assert torch.equal(mxq.gemm(a, w, u=wide, l2t=l2t.view(torch.int16)), want)
    y = mxq.gemm(a, w, u=u, l2t=l2t.flip(0).contiguous(), w_out_col=torch.cat([rev, rev]))
    assert torch.equal(y.flip(1), want)


# ---- quantized operands ----------------------------------------------------

def test_int8_operand_refuses_float8():
    a, _ = product()
    for dt in (torch.float8_e4m3fn, torch.float8_e5m2):
        with pytest.raises(ValueError):
            mxq.int8_operand(a.codes.view(dt), a.scales)


# what is wrong with codes or scales of 6 x 256 operands, by format
WRONG = [
    (mxq.INT8, "codes", lambda t: t.view(torch.float8_e4m3fn)), (mxq.INT8, "codes", lambda t: t.to(torch.int32)),
    (mxq.INT8, "codes", lambda t: t[:, :K - 16]), (mxq.INT8, "codes", lambda t: t.t().contiguous().t()),
    (mxq.INT8, "scales", lambda t: t.view(torch.int32)), (mxq.INT8, "scales", lambda t: t.to(torch.float64)),
    (mxq.INT8, "scales", lambda t: t.to(torch.float16)),
    (mxq.MXFP4, "codes", lambda t: t.to(BF16)), (mxq.MXFP4, "codes", lambda t: t[:, :K // 2 - 16]),
    (mxq.MXFP4, "codes", lambda t: t.repeat(1, 2)[:, ::2]), (mxq.MXFP4, "scales", lambda t: t.float()),
    (mxq.MXFP4, "scales", lambda t: t[:, :4]), (mxq.MXFP4, "scales", lambda t: t.flatten()),
    (mxq.NVFP4, "tensor_scale", lambda t: t.double()), (mxq.NVFP4, "tensor_scale", lambda t: t[:0]),
    (mxq.NVFP4, "scales", lambda t: t[:, :8]), (mxq.BF16, "codes", lambda t: t.to(torch.float16)),
    (mxq.BF16, "codes", lambda t: t[:, :K - 8]),
]


@pytest.mark.parametrize("case", range(len(WRONG)))
def test_operands_refuse(case):
    """As an operand of a product, and as what quantize writes."""
    fmt, name, spoil = WRONG[case]
    if fmt == mxq.BF16:
        a, w = mxq.bf16_operand(zeros(M, K, dtype=BF16)), product(mxq.MXFP4)[1]
    else:
        a, w = product(fmt)
    mxq.gemm(a, w)
    bad = mxq.QTensor(a.fmt, a.rows, a.cols, a.codes, a.scales, a.tensor_scale)
    setattr(bad, name, spoil(getattr(a, name)))
    with pytest.raises(ValueError):
        mxq.gemm(bad, w)
    if fmt in (mxq.INT8, mxq.MXFP4):
        with pytest.raises(ValueError):
            mxq.gemm_grouped(bad, w, torch.tensor([0, M], dtype=torch.int32, device="cuda"))
    if fmt != mxq.BF16:
        with pytest.raises(ValueError):
            mxq.gemm(a, mxq.QTensor(w.fmt, w.rows, w.cols, *[spoil(v) if n == name else v for n, v in
                                                             [("codes", w.codes), ("scales", w.scales),
                                                              ("tensor_scale", w.tensor_scale)]]))
        with pytest.raises(ValueError):
            mxq.quantize(zeros(M, K), fmt, out=bad)


def test_operands_take_bits_and_packed_types():
    """The same bytes under other types, and rows wider than the columns."""
    for fmt in (mxq.INT8, mxq.MXFP4, mxq.NVFP4, mxq.MXFP8, mxq.INT4):
        a, w = product(mxq.MXFP4 if fmt == mxq.INT4 else fmt)
        w = product(mxq.MXFP4)[1] if fmt == mxq.MXFP8 else product(fmt)[1]
        want = mxq.gemm(a, w)
        wide = torch.zeros(M, a.codes.shape[1] + 32, dtype=torch.uint8, device="cuda")
        wide[:, :a.codes.shape[1]] = a.codes
        assert torch.equal(mxq.gemm(mxq.QTensor(a.fmt, M, K, wide, a.scales, a.tensor_scale), w), want)
        if fmt == mxq.INT8:
            other = mxq.QTensor(a.fmt, M, K, a.codes.view(torch.int8), a.scales.flatten())
        else:
            other = mxq.QTensor(a.fmt, M, K, a.codes.view(torch.int32), a.scales.view(torch.int8), a.tensor_scale)
        assert torch.equal(mxq.gemm(other, w), want)
    x = torch.randn(M, K, device="cuda").to(BF16)
    w = product(mxq.MXFP4)[1]
    assert torch.equal(mxq.gemm(mxq.QTensor(mxq.BF16, M, K, x.view(torch.int16), None), w),
                       mxq.gemm(mxq.bf16_operand(x), w))


@pytest.mark.parametrize("fmt", [mxq.INT8, mxq.MXFP4, mxq.NVFP4, mxq.BF16])
def test_no_rows(fmt):
    """An empty batch: its tensors have no address, and it is a no-op."""
    a = mxq.bf16_operand(zeros(0, K, dtype=BF16)) if fmt == mxq.BF16 else mxq.quantize(zeros(0, K), fmt)
    w = product(mxq.MXFP4 if fmt == mxq.BF16 else fmt)[1]
    assert mxq.gemm(a, w).shape == (0, N)
    out = torch.full((4, N), 3.0, dtype=BF16, device="cuda")
    mxq.gemm(a, w, out=out)
    assert bool((out == 3).all())
    if fmt != mxq.NVFP4:
        off = torch.zeros(3, dtype=torch.int32, device="cuda")
        y = mxq.gemm_grouped(a, w, off)
        assert y.shape == (0, N // 2) and y.dtype == BF16


@pytest.mark.parametrize("dt", [torch.int16, torch.uint16, torch.float16])
@pytest.mark.parametrize("fmt", [mxq.INT8, mxq.MXFP4])
def test_out_and_bias_as_bits(fmt, dt):
    """out may be memory of any 16-bit type that the bf16 results are put into,
    bias bf16 bits of an integer type."""
    a, w = product(fmt)
    bias = torch.randn(N, device="cuda").to(BF16)
    off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    want = mxq.gemm(a, w, bias=bias)
    bits = bias if dt == torch.float16 else bias.view(dt)
    out = zeros(M, N, dtype=dt)
    assert mxq.gemm(a, w, bias=bits, out=out) is out and torch.equal(out.view(BF16), want)
    out = zeros(M, N, dtype=dt)
    mxq.gemm_grouped(a, w, off, bias=bits, out=out)
    assert torch.equal(out.view(BF16), mxq.gemm_grouped(a, w, off, bias=bias))
    with pytest.raises(ValueError):
        mxq.gemm(a, w, bias=bias.to(torch.float16))


@pytest.mark.parametrize("fmt", [mxq.INT8, mxq.MXFP4, mxq.BF16])
def test_one_row_operands_of_any_stride(fmt):
    """One token (and one output channel) as a transposed column, an expanded
    row and a row of a strided view."""
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.randn(1, K, generator=g, device="cuda").to(BF16)
    a = mxq.bf16_operand(x) if fmt == mxq.BF16 else mxq.quantize(x, fmt)
    w = product(mxq.MXFP4 if fmt == mxq.BF16 else fmt)[1]
    w1 = mxq.QTensor(w.fmt, 1, K, w.codes[:1], w.scales[:1])
    off = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    want, want1 = mxq.gemm(a, w), mxq.gemm(a, w1)

    def forms(t):
        if t is None:
            return [None] * 3
        return [t.reshape(-1, 1).contiguous().t(), t[0].expand(1, -1),
                torch.cat([t] * 3)[::3] if t.shape[1] > 1 else t.expand(1, 1)]

    for codes, scales in zip(forms(a.codes), forms(a.scales)):
        one = mxq.QTensor(a.fmt, 1, K, codes, scales)
        assert torch.equal(mxq.gemm(one, w), want) and torch.equal(mxq.gemm_grouped(one, w, off), want)
    for codes, scales in zip(forms(w1.codes), forms(w1.scales)):
        assert torch.equal(mxq.gemm(a, mxq.QTensor(w.fmt, 1, K, codes, scales)), want1)
