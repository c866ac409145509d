"""CPU checks of the FP8, gated and layer-norm entry points: storage sizes and
refusals (every call stops before any device work; the pointers are stand-ins
that are never read)."""
import ctypes as C

import pytest

from fp8_quantized_linear_mxq_amd import _lib

vp = C.c_void_p
INV, UNSUP, ALIGN, SHAPE, WS = 1, 2, 3, 4, 5


def f8(rows, cols, ld=None, codes=4096, scales=8192, lds=None):
    return _lib.QTensorC(7, 0, rows, cols, vp(codes), (cols + 15) // 16 * 16 if ld is None else ld, vp(scales),
                         4 * rows if lds is None else lds, None)


def f8t(rows, cols, ld=None, codes=4096, scales=8192, lds=None):
    return _lib.QTensorC(8, 0, rows, cols, vp(codes), (cols + 15) // 16 * 16 if ld is None else ld, vp(scales),
                         (cols + 127) // 128 * 4 if lds is None else lds, None)


def bf(rows, cols, ld=None):
    return _lib.QTensorC(5, 0, rows, cols, vp(4096), 2 * cols if ld is None else ld, None, 0, None)


def mx4(rows, cols):
    return _lib.QTensorC(1, 0, rows, cols, vp(4096), (cols // 2 + 15) // 16 * 16, vp(8192), (cols // 32 + 3) // 4 * 4, None)


def test_storage_and_workspaces(lib):
    assert _lib.storage(_lib.FP8, 96) == (96, 4) and _lib.storage(_lib.FP8, 1184) == (1184, 40)
    assert _lib.storage(_lib.FP8_TILE, 256) == (256, 8)
    with pytest.raises(_lib.MxqError):
        _lib.storage(_lib.FP8, 40)
    assert _lib.workspace_size(_lib.OP_QUANTIZE, 10, 64, _lib.FP8) == 0
    assert _lib.workspace_size(_lib.OP_GEMM, 10, 64, _lib.FP8_TILE) == 0
    assert _lib.workspace_size(_lib.OP_QUANTIZE_MSE, 10, 64, _lib.FP8) == -1
    size = _lib.workspace_size
    assert size(_lib.OP_GATED_BACKWARD, 64, 64) == 64 * 128 * 2 and size(_lib.OP_GATED_BACKWARD, 65, 1) == 128 * 128 * 2
    assert size(_lib.OP_GATED_BACKWARD, 0, 10) == 0 and size(_lib.OP_GATED_BACKWARD, 1 << 31, 8) == -1
    # few rows and a long sum: room for the split sums; many tiles: none
    assert size(_lib.OP_GATED_BACKWARD, 64, 4096, 512) > size(_lib.OP_GATED_BACKWARD, 64, 4096)
    assert size(_lib.OP_GATED_BACKWARD, 8192, 8192, 8192) == size(_lib.OP_GATED_BACKWARD, 8192, 8192)
    assert size(_lib.OP_LAYER_NORM_BACKWARD, 5, 100) == 256 * 2 * 100 * 4
    assert size(_lib.OP_LAYER_NORM_BACKWARD, 5, (1 << 26) + 1) == -1


def test_quantize_refusals(lib):
    def call(q, rows=4, cols=64, x=16, dt=1, had=0, rank=0, l1=None, u=None):
        return lib.mxq_quantize(vp(x), dt, rows, cols, cols, had, None, l1, rank, u, 32, C.byref(q), None, 0, None)
    for make in (f8, f8t):
        assert call(make(4, 48), cols=48) == SHAPE
        assert call(make(4, 64, ld=48)) == INV
        assert call(make(4, 64, ld=72)) == ALIGN
        assert call(make(4, 64, lds=18)) in (ALIGN, INV)
        assert call(make(4, 64), x=20) == ALIGN
        assert call(make(4, 96), cols=96, had=128) == SHAPE
        assert call(make(4, 128), cols=128, dt=2, rank=16, l1=vp(32), u=vp(64)) == UNSUP   # no low-rank projection
        assert call(make(0, 64), rows=0) == 0
        q = make(4, 64)
        assert lib.mxq_quantize_mse(vp(16), 1, 4, 64, 64, C.byref(q), None, 0, None) == UNSUP
    assert call(f8(8, 64, lds=28), rows=8) == INV            # a K-block holds every row's scale
    assert call(f8t(4, 256, lds=4), cols=256) == INV


def test_gemm_refusals(lib):
    def call(a, w, out=64, ld=8, n=8, rank=0, u=None, l2=None):
        return lib.mxq_gemm(C.byref(a), C.byref(w), None, u, 32, l2, rank, None, vp(out), ld, n, None, 0, None)
    assert call(f8(8, 128), f8(8, 128)) == UNSUP             # rows go with tiles only
    assert call(f8t(8, 128), f8t(8, 128)) == UNSUP
    assert call(f8(8, 128), mx4(8, 128)) == UNSUP
    assert call(mx4(8, 128), f8t(8, 128)) == UNSUP
    assert call(bf(8, 128), f8t(8, 128)) == UNSUP
    assert call(f8(8, 128), f8t(8, 128), rank=16, u=vp(64), l2=vp(64)) == UNSUP
    assert call(f8(8, 128), f8t(8, 160)) == SHAPE
    assert call(f8(8, 0), f8t(8, 0)) == SHAPE
    assert call(f8(8, 96, ld=(1 << 24) + 16), f8t(8, 96)) == SHAPE
    assert call(f8(8, 96), f8t(9, 96)) == SHAPE
    assert call(f8(8, 96), f8t(8, 96), ld=7) == INV
    assert call(f8(0, 96), f8t(8, 96)) == 0
    x, w = f8(20, 128), f8t(8, 1152)
    assert lib.mxq_conv3x3_gemm_mixed(C.byref(x), 4, 5, C.byref(w), 1, None, None, vp(64), 8, 8, None, 0, None) == UNSUP
    x8 = _lib.QTensorC(2, 0, 20, 128, vp(4096), 128, vp(8192), 4, None)
    assert lib.mxq_conv3x3_gemm_mixed(C.byref(x8), 4, 5, C.byref(w), 1, None, None, vp(64), 8, 8, None, 0, None) == UNSUP

    def grouped(a, w, e=4, ld=128):
        return lib.mxq_gemm_grouped(C.byref(a), C.byref(w), e, vp(64), None, vp(64), ld, None)
    assert grouped(f8(8, 128), f8t(4 * 64, 128)) == SHAPE    # a tile would span two experts
    assert grouped(f8(8, 128), mx4(4 * 128, 128)) == UNSUP
    assert grouped(f8(8, 128), f8t(4 * 128, 128), ld=127) == INV
    assert grouped(f8(8, 0), f8t(4 * 128, 0)) == SHAPE
    assert grouped(f8(0, 128), f8t(4 * 128, 128)) == 0


def test_gated_refusals(lib):
    def call(x, g, u, act=1, saved=None, out=64, ld=8):
        return lib.mxq_gemm_gated(C.byref(x), C.byref(g), C.byref(u), act, vp(saved), vp(out), ld, None)
    assert call(bf(4, 64), bf(8, 64), f8t(8, 64)) == UNSUP
    assert call(bf(4, 64), f8t(8, 64), f8t(8, 64)) == UNSUP
    assert call(f8(4, 64), bf(8, 64), bf(8, 64)) == UNSUP
    assert call(f8(4, 64), f8(8, 64), f8(8, 64)) == UNSUP
    assert call(mx4(4, 64), mx4(8, 64), mx4(8, 64)) == UNSUP
    assert call(f8(4, 64), f8t(8, 64), f8t(8, 64), saved=4096) == UNSUP      # nothing to differentiate
    for act in (0, 4, -1):
        assert call(bf(4, 64), bf(8, 64), bf(8, 64), act=act) == INV
    assert call(bf(4, 64), bf(8, 72), bf(8, 64)) == SHAPE
    assert call(bf(4, 64), bf(8, 64), bf(9, 64)) == SHAPE
    assert call(bf(4, 68, ld=144), bf(8, 68, ld=144), bf(8, 68, ld=144)) == SHAPE   # K a multiple of 8
    assert call(bf(4, 64, ld=136), bf(8, 64), bf(8, 64)) == ALIGN
    assert call(bf(4, 64, ld=(1 << 24) + 16), bf(8, 64), bf(8, 64)) == SHAPE
    assert call(bf(4, 64), bf(8, 64), bf(8, 64), ld=7) == INV
    assert call(bf(4, 64), bf(8, 64), bf(8, 64), out=None) == INV
    assert call(bf(4, 64), bf(8, 64), bf(8, 64), out=65) == ALIGN
    assert call(bf(4, 64), bf(8, 64), bf(8, 64), saved=4098) == ALIGN
    assert call(bf(4, 0), bf(8, 0), bf(8, 0)) == SHAPE
    assert call(bf(0, 64), bf(8, 64), bf(8, 64), out=None) == 0
    assert call(bf(4, 64), bf(0, 64), bf(0, 64), out=None) == 0

    base = dict(dy=64, ld_dy=8, x=bf(4, 64), g=bf(8, 64), u=bf(8, 64), act=1, saved=64, dx=64, ld_dx=64, dg=64, du=64,
                ld_dw=64, ws=4096, wsb=1 << 20)

    def back(**o):
        a = dict(base, **o)
        return lib.mxq_gemm_gated_backward(vp(a["dy"]), a["ld_dy"], C.byref(a["x"]), C.byref(a["g"]), C.byref(a["u"]), a["act"],
                                           vp(a["saved"]), vp(a["dx"]), a["ld_dx"], vp(a["dg"]), vp(a["du"]), a["ld_dw"],
                                           vp(a["ws"]), a["wsb"], None)
    assert back(x=f8(4, 64), g=f8t(8, 64), u=f8t(8, 64)) == UNSUP
    assert back(act=9) == INV
    assert back(dg=None) == INV                              # both or neither
    assert back(dy=None) == INV
    assert back(ld_dy=7) == INV
    assert back(saved=None) == INV
    assert back(ld_dx=63) == INV
    assert back(ld_dw=63) == INV
    assert back(dx=65) == ALIGN
    assert back(du=65) == ALIGN
    assert back(saved=66) == ALIGN
    assert back(ws=None) == WS
    assert back(ws=4104) == WS
    assert back(wsb=64 * 128 * 2 - 1) == WS
    assert back(dx=None, dg=None, du=None, ws=None) == 0     # nothing asked for


def test_layer_norm_refusals(lib):
    base = dict(x=64, dt=2, rows=4, cols=9, ldx=9, w=64, b=64, eps=1e-5, y=64, ldy=9, stats=64)

    def call(**o):
        a = dict(base, **o)
        return lib.mxq_layer_norm(vp(a["x"]), a["dt"], a["rows"], a["cols"], a["ldx"], vp(a["w"]), vp(a["b"]), a["eps"],
                                  vp(a["y"]), a["ldy"], vp(a["stats"]), None)
    assert call(dt=3) == INV
    assert call(eps=-1.0) == INV
    assert call(eps=float("nan")) == INV
    assert call(rows=-1) == INV
    assert call(x=None) == INV
    assert call(y=None) == INV
    assert call(ldx=8) == INV
    assert call(ldy=8) == INV
    assert call(cols=(1 << 26) + 1, ldx=1 << 27, ldy=1 << 27) == SHAPE
    assert call(rows=1 << 31) == SHAPE
    assert call(x=65) == ALIGN
    assert call(dt=1, w=66) == ALIGN
    assert call(b=65) == ALIGN
    assert call(stats=68) == ALIGN
    assert call(rows=0, x=None, y=None) == 0
    assert call(cols=0) == 0

    base2 = dict(dy=64, ld_dy=9, x=64, dt=2, rows=4, cols=9, ldx=9, stats=64, w=64, dx=64, ld_dx=9, dw=64, db=64, ws=4096,
                 wsb=256 * 2 * 9 * 4)

    def back(**o):
        a = dict(base2, **o)
        return lib.mxq_layer_norm_backward(vp(a["dy"]), a["ld_dy"], vp(a["x"]), a["dt"], a["rows"], a["cols"], a["ldx"],
                                           vp(a["stats"]), vp(a["w"]), vp(a["dx"]), a["ld_dx"], vp(a["dw"]), vp(a["db"]),
                                           vp(a["ws"]), a["wsb"], None)
    assert back(dt=0) == INV
    assert back(cols=-1) == INV
    assert back(dy=None) == INV
    assert back(x=None) == INV
    assert back(stats=None) == INV
    assert back(ld_dy=8) == INV
    assert back(ld_dx=8) == INV
    assert back(stats=68) == ALIGN
    assert back(dw=65) == ALIGN
    assert back(dx=65) == ALIGN
    assert back(ws=None) == WS
    assert back(wsb=256 * 2 * 9 * 4 - 1) == WS
    assert back(rows=0, dw=None, db=None) == 0
    assert back(dx=None, dw=None, db=None, dy=None) == 0


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    import fp8_quantized_linear_mxq_amd as mxq
    codes, s = torch.zeros((4, 160), dtype=torch.uint8), torch.zeros((2, 4))
    q = mxq.fp8_operand(codes, s).c()
    assert (q.fmt, q.rows, q.cols, q.ld_codes, q.ld_scales) == (7, 4, 160, 160, 16)
    q = mxq.fp8_operand(codes.view(torch.float8_e4m3fn), torch.zeros((1, 2)), tile=True).c()
    assert (q.fmt, q.ld_codes, q.ld_scales) == (8, 160, 8)
    for c, t, tile in ((codes.short(), s, False), (codes[0], s, False), (codes.t(), s, False), (codes, s.double(), False),
                       (codes, s.t(), False), (codes, s, True), (codes, s[:, :3], False),
                       (codes.view(torch.float8_e5m2), s, False), (codes.bool(), s, False)):
        with pytest.raises(ValueError):
            mxq.fp8_operand(c, t, tile=tile)
    x, w = torch.zeros((4, 16), dtype=torch.bfloat16), torch.zeros((8, 16), dtype=torch.bfloat16)
    ops = [mxq.bf16_operand(t) for t in (x, w, w)]
    with pytest.raises(ValueError):                          # host memory
        mxq.gemm_gated(*ops)
    with pytest.raises(ValueError):
        mxq.gemm_gated_backward(torch.zeros((4, 8), dtype=torch.bfloat16), *ops, torch.zeros((2, 4, 8)))
    for fn in (lambda: mxq.layer_norm(x), lambda: mxq.layer_norm_backward(x, x, torch.zeros((4, 2)))):
        with pytest.raises(ValueError):
            fn()


def test_no_gradients_through_autograd_in_a_capture(monkeypatch):
    torch = pytest.importorskip("torch")
    import fp8_quantized_linear_mxq_amd as mxq
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    x, w = torch.zeros((4, 16), dtype=torch.bfloat16), torch.zeros((8, 16), dtype=torch.bfloat16, requires_grad=True)
    with pytest.raises(RuntimeError, match="gemm_gated_backward"):
        mxq.autograd.gated(x, w, w)
    with pytest.raises(RuntimeError, match="layer_norm_backward"):
        mxq.autograd.layer_norm(x, w[0])
    with torch.no_grad(), pytest.raises(ValueError):         # goes on to the call, which refuses host memory
        mxq.autograd.layer_norm(x, w[0])
