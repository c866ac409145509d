"""CPU checks of the int8, grouped and head-norm entry points: storage sizes
and refusals (every call stops before any device work; the pointers are
stand-ins that are never read)."""
import ctypes as C

import pytest

from fp8_quantized_linear_mxq_amd import _lib

vp = C.c_void_p
INV, UNSUP, ALIGN, SHAPE = 1, 2, 3, 4


def i8(rows, cols, ld=None, codes=4096, scales=8192, lds=4):
    return _lib.QTensorC(6, 0, rows, cols, vp(codes), cols if ld is None else ld, vp(scales), lds, None)


def mx4(rows, cols):
    return _lib.QTensorC(1, 0, rows, cols, vp(4096), (cols // 2 + 15) // 16 * 16, vp(8192),
                         (cols // 32 + 3) // 4 * 4, None)


def bf(rows, cols):
    return _lib.QTensorC(5, 0, rows, cols, vp(4096), 2 * cols, None, 0, None)


def test_storage(lib):
    assert _lib.storage(_lib.INT8, 96) == (96, 4)
    with pytest.raises(_lib.MxqError):
        _lib.storage(_lib.INT8, 40)
    assert _lib.workspace_size(_lib.OP_QUANTIZE, 10, 64, _lib.INT8) == 0
    assert _lib.workspace_size(_lib.OP_GEMM, 10, 64, _lib.INT8) == 0
    assert _lib.workspace_size(_lib.OP_QUANTIZE_MSE, 10, 64, _lib.INT8) == -1


def test_quantize_refusals(lib):
    def call(q, rows=4, cols=64, x=16, dt=1, had=0, rank=0, fn=lib.mxq_quantize, l1=None, u=None):
        return fn(vp(x), dt, rows, cols, cols, had, None, l1, rank, u, 32, C.byref(q), None, 0, None)
    assert call(i8(4, 48), cols=48) == SHAPE                 # not a multiple of 32
    assert call(i8(4, 64, lds=2)) == INV                     # no room for a scale
    assert call(i8(4, 64, lds=6)) == ALIGN
    assert call(i8(4, 64, ld=72)) == ALIGN
    assert call(i8(4, 64), x=20) == ALIGN
    assert call(i8(4, 96), cols=96, had=128) == SHAPE
    assert call(i8(0, 64), rows=0) == 0                      # empty
    # the packed low-rank factor is read by the block formats' kernel only
    assert call(i8(4, 128), cols=128, dt=2, rank=16, fn=lib.mxq_quantize_lrp, l1=vp(32), u=vp(64)) == UNSUP
    # not a least-squared-error format, not a selection candidate
    q = i8(4, 64)
    assert lib.mxq_quantize_mse(vp(16), 1, 4, 64, 64, C.byref(q), None, 0, None) == UNSUP
    cand = (C.c_int32 * 1)(6)
    assert lib.mxq_select_format(vp(16), 1, 4, 64, 64, cand, 1, vp(64), None, None, None, None, None, 0,
                                 None) == UNSUP


def test_gemm_refusals(lib):
    def call(a, w, out=64, ld=8, n=8):
        return lib.mxq_gemm(C.byref(a), C.byref(w), None, None, 0, None, 0, None, vp(out), ld, n, None, 0, None)
    assert call(i8(8, 128), mx4(8, 128)) == UNSUP            # int8 pairs with int8 only
    assert call(mx4(8, 128), i8(8, 128)) == UNSUP
    assert call(bf(8, 128), i8(8, 128)) == UNSUP
    assert call(i8(8, 128), i8(8, 160)) == SHAPE
    assert call(i8(8, 0), i8(8, 0)) == SHAPE
    big = (1 << 17) + 32                                     # sums would leave int32
    assert call(i8(8, big), i8(8, big)) == SHAPE
    assert call(i8(8, 96, ld=(1 << 24) + 16), i8(8, 96)) == SHAPE
    assert call(i8(8, 96), i8(8, 96), ld=7) == INV
    assert call(i8(8, 96), i8(9, 96)) == SHAPE               # more rows than columns out, no map
    assert call(i8(0, 96), i8(8, 96)) == 0
    x = i8(20, 128)
    w = i8(8, 1152)
    assert lib.mxq_conv3x3_gemm_mixed(C.byref(x), 4, 5, C.byref(w), 1, None, None, vp(64), 8, 8, None, 0,
                                      None) == UNSUP
    two = (_lib.QTensorC * 2)(i8(4, 128), mx4(4, 128))
    a = i8(8, 128)
    assert lib.mxq_gemm_mixed(C.byref(a), two, 2, vp(64), None, 0, None, 0, None, vp(64), 8, 8, None, 0,
                              None) == UNSUP


def test_grouped_refusals(lib):
    def call(a, w, e=4, off=64, out=64, ld=8):
        return lib.mxq_gemm_grouped(C.byref(a), C.byref(w), e, vp(off), None, vp(out), ld, None)
    assert call(i8(8, 128), i8(32, 128), e=0) == INV
    assert call(i8(8, 128), i8(32, 128), e=65537) == INV
    assert call(i8(8, 128), i8(30, 128)) == SHAPE            # rows not whole experts
    assert call(i8(8, 128), i8(32, 256)) == SHAPE
    assert call(mx4(8, 128), i8(32, 128)) == UNSUP
    assert call(i8(8, 128), mx4(32, 128)) == UNSUP
    assert call(mx4(8, 192), mx4(32, 192)) == SHAPE          # 4-bit: K a multiple of 128
    mx8 = _lib.QTensorC(2, 0, 8, 128, vp(4096), 128, vp(8192), 4, None)
    assert call(mx8, mx4(32, 128)) == UNSUP
    assert call(i8(8, 128), i8(32, 128), off=None) == INV
    assert call(i8(8, 128), i8(32, 128), out=None) == INV
    assert call(i8(8, 128), i8(32, 128), ld=7) == INV
    assert call(i8(8, 128), i8(32, 128), off=66) == ALIGN
    assert call(i8(8, 0), i8(32, 0)) == SHAPE
    assert call(i8(0, 128), i8(32, 128), off=None, out=None) == 0
    assert call(i8(8, 128), i8(0, 128), off=None, out=None) == 0
    bad = i8(8, 128)
    bad.reserved = 1
    assert call(bad, i8(32, 128)) == INV


def test_head_norm_refusals(lib):
    base = dict(x=4096, dt=2, tokens=4, ldx=256, nq=2, nk=1, d=64, wq=None, wk=None, eps=1e-6, cos=8192,
                sin=8192, npos=8, rot=64, inter=0, pos=None, q=16384, qt=128, qh=64, k=32768, kt=64, kh=64)

    def call(**o):
        a = dict(base, **o)
        return lib.mxq_qk_norm_rope(vp(a["x"]), a["dt"], a["tokens"], a["ldx"], a["nq"], a["nk"], a["d"],
                                    vp(a["wq"]), vp(a["wk"]), a["eps"], vp(a["cos"]), vp(a["sin"]), a["npos"],
                                    a["rot"], a["inter"], vp(a["pos"]), vp(a["q"]), a["qt"], a["qh"],
                                    vp(a["k"]), a["kt"], a["kh"], None)
    assert call(dt=3) == INV
    assert call(d=0) == INV
    assert call(rot=72) == INV                               # more than the head
    assert call(rot=-8) == INV
    assert call(inter=2) == INV
    assert call(eps=-1.0) == INV
    assert call(eps=float("nan")) == INV
    assert call(d=60, rot=56) == SHAPE
    assert call(d=520, ldx=4096) == SHAPE
    assert call(rot=60) == SHAPE
    assert call(ldx=184) == INV                              # narrower than the heads
    assert call(x=None) == INV
    assert call(cos=None) == INV
    assert call(npos=3) == SHAPE                             # token 3 has no position
    assert call(q=None) == INV
    assert call(k=None) == INV
    assert call(x=4104) == ALIGN
    assert call(ldx=196) == ALIGN
    assert call(wq=4104) == ALIGN
    assert call(sin=8196) == ALIGN
    assert call(pos=66, npos=1) == ALIGN
    assert call(q=16392) == ALIGN
    assert call(kt=68) == ALIGN
    assert call(tokens=0, x=None) == 0
    assert call(nq=0, nk=0, x=None) == 0


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    import fp8_quantized_linear_mxq_amd as mxq
    codes, s = torch.zeros((4, 32), dtype=torch.int8), torch.zeros(4)
    q = mxq.int8_operand(codes, s[:, None]).c()
    assert (q.fmt, q.rows, q.cols, q.ld_codes, q.ld_scales) == (6, 4, 32, 32, 4)
    for c, t in ((codes.short(), s), (codes[0], s), (codes.t(), s), (codes, s.double()), (codes, s[:3])):
        with pytest.raises(ValueError):
            mxq.int8_operand(c, t)
    a = mxq.int8_operand(codes, s)
    with pytest.raises(ValueError):
        mxq.gemm_grouped(a, a, torch.zeros(3, dtype=torch.int64))
    x = torch.zeros((2, 96), dtype=torch.bfloat16)
    tab = torch.zeros((2, 16))
    for kw in (dict(x=x.half()), dict(x=x.t()), dict(n_q_heads=4), dict(q_weight=torch.zeros(32)),
               dict(q_weight=torch.zeros(16, dtype=torch.bfloat16)), dict(cos=tab, sin=tab.half()),
               dict(cos=tab, sin=None), dict(cos=tab, sin=tab[:, :8]),
               dict(cos=tab, sin=tab, positions=torch.zeros(2, dtype=torch.int64)),
               dict(q_out=torch.zeros((2, 2, 32)))):
        args = dict(dict(x=x, n_q_heads=2, n_k_heads=1, head_dim=32), **kw)
        with pytest.raises(ValueError):
            mxq.qk_norm_rope(**args)
