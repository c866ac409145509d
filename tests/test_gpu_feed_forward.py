"""The FP8, gated and layer-norm operators together: the block of
examples/feed_forward.py, trained and served; autograd; captured graphs,
streams, refusals of the binding, offsets that pass 32 bits."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import fp8_quantized_linear_mxq_amd as mxq
from fp8_quantized_linear_mxq_amd import _lib
from oracle import feed_forward as ff
from oracle import fp8 as o8
from tests import gpu_util as gu
from tests.test_gpu_fp8 import bf16, gen
from tests.test_gpu_gated import exact_case

pytestmark = pytest.mark.gpu

_path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "feed_forward.py")
_spec = importlib.util.spec_from_file_location("feed_forward", _path)
ex = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(ex)

BF, F32 = torch.bfloat16, torch.float32


def _np(t):
    return t.detach().double().cpu().numpy()


def distance(got, want):
    return float(np.linalg.norm(_np(got) - want) / np.linalg.norm(want))


# ---- the block -------------------------------------------------------------

def block(width, hidden, act, seed):
    b = ex.FeedForward(width, hidden, act, seed)
    g = gen(seed + 1)
    with torch.no_grad():
        b.gain.copy_(1 + 0.2 * torch.randn(width, generator=g, device="cuda"))
        b.shift.copy_(0.3 * torch.randn(width, generator=g, device="cuda"))
    return b


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("tokens,width,hidden", [(1, 64, 200), (37, 256, 704), (300, 512, 1000)])
def test_block_gradients(tokens, width, hidden, act):
    """Against the same block in float64.  Between an output or gradient and its
    exact value lie at most eight roundings to bf16 (norm, gated product, down
    product; the gradients of the three, dg and du, the result), 2**-8 relative
    each; through linear maps their relative sizes in the 2-norm stay."""
    gu.say(f"block {tokens}x{width}x{hidden} {act}")
    b = block(width, hidden, act, tokens)
    g = gen(tokens + 7)
    x = torch.randn((tokens, width), generator=g, device="cuda").bfloat16().requires_grad_()
    dy = torch.randn((tokens, width), generator=g, device="cuda").bfloat16()
    y = b(x)
    grads = torch.autograd.grad(y, [x, b.gain, b.shift, b.gate, b.up, b.down], dy)
    xn, dn, wn, sn, gn, un, on = (_np(t) for t in (x, dy, b.gain, b.shift, b.gate, b.up, b.down))
    h, _, _ = ff.layer_norm(xn, wn, sn)
    p, _, _ = ff.gated(h, gn, un, act)
    assert distance(y, xn + p @ on.T) <= 8 * 2.0 ** -8
    dh, dgate, dup, _, _ = ff.gated_backward(dn @ on, h, gn, un, act)
    dx, dw, db = ff.layer_norm_backward(dh, xn, wn)
    for name, got, want in zip("x gain shift gate up down".split(), grads, (dn + dx, dw, db, dgate, dup, dn.T @ p)):
        assert got.shape == want.shape and distance(got, want) <= 8 * 2.0 ** -8, name


@pytest.mark.parametrize("tokens,width,hidden", [(1, 256, 704), (50, 512, 1408), (600, 256, 1024)])
def test_block_on_codes(tokens, width, hidden):
    """Against float64 from the dequantized weights.  The bf16 roundings before a
    quantize (two, 2**-9 at the middle of a step) move a code of step d (relative;
    E4M3: 2**-4 to 2**-3) to its neighbour with probability 2**-8 / d, an rms of
    sqrt(2**-8 d) <= 2.3 %, in each of the two quantizes; sums of many such are
    independent, together 3.2 %."""
    gu.say(f"block on codes {tokens}x{width}x{hidden}")
    b = block(width, hidden, "silu", tokens)
    q = ex.QuantizedFeedForward(b)
    x = torch.randn((tokens, width), generator=gen(tokens), device="cuda").bfloat16()
    y = q(x)
    dense = lambda t: o8.dequantize(t.codes.view(torch.uint8).cpu().numpy()[:, :t.cols], t.scales.cpu().numpy(), True)   # noqa: E731
    codes = lambda v: o8.dequantize(*o8.quantize(v.astype(np.float32)))   # noqa: E731
    xn = _np(x)
    h, _, _ = ff.layer_norm(xn, _np(q.gain), _np(q.shift))
    p, _, _ = ff.gated(codes(h), dense(q.gate), dense(q.up), "silu")
    assert distance(y.float() - x.float(), codes(p) @ dense(q.down).T) <= 0.032


def test_example_runs(capsys, monkeypatch):
    monkeypatch.setattr("sys.argv", ["feed_forward.py", "--tokens", "40", "--width", "128", "--hidden", "256", "--steps", "2"])
    ex.main()
    assert "2 steps" in capsys.readouterr().out


# ---- autograd --------------------------------------------------------------

def test_autograd_is_the_operators():
    """Leading dimensions, strided and broadcast inputs; the library's own bits."""
    g = gen(3)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()   # noqa: E731
    wide, wg, wu = r(3, 9, 96), r(70, 64), r(70, 64)
    x = wide[:, 2:7, :64].requires_grad_()
    for t in (wg, wu):
        t.requires_grad_()
    y = mxq.autograd.gated(x, wg, wu, "gelu")
    flat = x.detach().reshape(15, 64)
    ops = [mxq.bf16_operand(t.detach()) for t in (flat, wg, wu)]
    saved = torch.empty((2, 15, 70), device="cuda")
    assert y.shape == (3, 5, 70) and torch.equal(y.detach().view(15, 70), mxq.gemm_gated(*ops, act="gelu", saved=saved))
    want = mxq.gemm_gated_backward(torch.ones_like(y).view(15, 70), *ops, saved, act="gelu")
    got = torch.autograd.grad(y.sum(), [x, wg, wu])          # the sum's gradient is one number, broadcast
    assert torch.equal(got[0].reshape(15, 64), want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])

    w, b = r(96).requires_grad_(), r(96).requires_grad_()
    x = wide.transpose(0, 1).requires_grad_()
    y = mxq.autograd.layer_norm(x, w, b, 1e-3)
    flat = x.detach().reshape(27, 96)
    stats = torch.empty((27, 2), device="cuda")
    assert torch.equal(y.detach().view(27, 96), mxq.layer_norm(flat, w.detach(), b.detach(), eps=1e-3, stats=stats))
    dy = r(9, 1, 96).expand(9, 3, 96)
    want = mxq.layer_norm_backward(dy.reshape(27, 96), flat, stats, w.detach())
    got = torch.autograd.grad(y, [x, w, b], dy)
    assert torch.equal(got[0].reshape(27, 96), want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])


def test_autograd_partial_and_empty():
    g = gen(4)
    x, wg, wu = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((6, 32), (40, 32), (40, 32)))
    with torch.no_grad():
        assert not mxq.autograd.gated(x, wg.requires_grad_(), wu).requires_grad
    y = mxq.autograd.gated(x, wg, wu)
    full = torch.autograd.grad(y, wg, torch.ones_like(y))[0]
    y = mxq.autograd.gated(x, wg, wg)                        # one leaf in both places
    assert torch.autograd.grad(y, wg, torch.ones_like(y))[0].shape == full.shape
    y = mxq.autograd.gated(x.requires_grad_(), wg.detach(), wu)
    y.sum().backward()
    assert x.grad.shape == (6, 32) and wu.grad is None
    for rows in (0, 1):
        x = torch.ones((rows, 32), device="cuda", requires_grad=True)
        w = torch.ones(32, device="cuda", requires_grad=True)
        y = mxq.autograd.layer_norm(x, w)
        dx, dw = torch.autograd.grad(y, [x, w], torch.ones_like(y))
        assert dx.shape == (rows, 32) and not bool(dw.any())  # a constant row's h is zero
    x = torch.ones((5, 1), device="cuda", requires_grad=True)
    assert not bool(torch.autograd.grad(mxq.autograd.layer_norm(x).sum(), x)[0].any())
    with pytest.raises(RuntimeError):                        # no gradients of gradients
        d = torch.autograd.grad(mxq.autograd.layer_norm(x).square().sum(), x, create_graph=True)[0]
        torch.autograd.grad(d.sum(), x)


def test_layer_norm_against_differences():
    """<dx, v> against (L(x + h v) - L(x - h v)) / 2h of L = <dy, y>, fp32.  The
    difference's own distance from the slope comes from the same difference in
    float64; each y is off by at most 2**-20 (|y| + |w|)."""
    g = gen(9)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")   # noqa: E731
    x, w, b, dy, v, h = r(5, 300), r(300), r(300), r(5, 300), r(5, 300), 2.0 ** -7
    stats = torch.empty((5, 2), device="cuda")
    mxq.layer_norm(x, w, b, stats=stats)
    dx = mxq.layer_norm_backward(dy, x, stats, w)[0]
    xs = [x + h * v, x - h * v]
    at = [_np(mxq.layer_norm(t, w, b)) for t in xs]
    ref = [ff.layer_norm(_np(t), _np(w), _np(b))[0] for t in xs]
    slope = (_np(xs[0]) - _np(xs[1])) / (2 * h)              # v as the rounded points have it
    dn = _np(dy)
    rx = ff.layer_norm_backward(dn, _np(x), _np(w))[0]
    truncation = abs((dn * (ref[0] - ref[1])).sum() / (2 * h) - (rx * slope).sum())
    rounding = sum((np.abs(dn) * 2.0 ** -20 * (np.abs(y) + np.abs(_np(w)))).sum() for y in ref) / (2 * h)
    assert truncation < 0.02 * abs((rx * slope).sum()) + 0.1
    assert abs((dn * (at[0] - at[1])).sum() / (2 * h) - (_np(dx) * slope).sum()) <= truncation + rounding + 2.0 ** -18 * np.abs(rx * slope).sum()


# ---- graphs and streams ----------------------------------------------------

def serve(x, w, parts):
    gain, shift, gate, up, down = w
    h = mxq.quantize(mxq.layer_norm(x, gain, shift, out=parts and parts[0]), mxq.FP8, out=parts and parts[1])
    y = mxq.quantize(mxq.gemm_gated(h, gate, up, out=parts and parts[2]), mxq.FP8, out=parts and parts[3])
    return mxq.gemm(y, down, out=parts and parts[4])


@pytest.mark.parametrize("tokens", [1, 20, 300])
@pytest.mark.parametrize("given", [False, True], ids=["allocated", "given"])
def test_served_block_in_a_graph(tokens, given):
    gu.say(f"graph of the served block, {tokens} tokens")
    width, hidden = 256, 640
    b = block(width, hidden, "silu", 5)
    q = ex.QuantizedFeedForward(b)
    w = (q.gain, q.shift, q.gate, q.up, q.down)
    x = torch.zeros((tokens, width), dtype=BF, device="cuda")
    parts = None
    if given:
        parts = [torch.empty((tokens, width), dtype=BF, device="cuda"), mxq.empty_qtensor(mxq.FP8, tokens, width),
                 torch.empty((tokens, hidden), dtype=BF, device="cuda"), mxq.empty_qtensor(mxq.FP8, tokens, hidden),
                 torch.empty((tokens, width), dtype=BF, device="cuda")]
    serve(x, w, parts)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = serve(x, w, parts)
    for rep in range(4):
        x.copy_(torch.randn((tokens, width), generator=gen(rep), device="cuda"))
        want = serve(x, w, None)
        y.fill_(-3)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), rep


def step(x, dy, gain, shift, wg, wu, ws):
    rows = x.shape[0]
    stats, saved = torch.empty((rows, 2), device="cuda"), torch.empty((2, rows, wg.shape[0]), device="cuda")
    h = mxq.layer_norm(x, gain, shift, stats=stats)
    ops = [mxq.bf16_operand(t) for t in (h, wg, wu)]
    y = mxq.gemm_gated(*ops, saved=saved)
    dh, dg, du = mxq.gemm_gated_backward(dy, *ops, saved, workspace=ws and ws[0])
    return (y, dg, du) + tuple(mxq.layer_norm_backward(dh, x, stats, gain, workspace=ws and ws[1]))


@pytest.mark.parametrize("rows", [1, 70, 700])
@pytest.mark.parametrize("given", [False, True], ids=["allocated", "given"])
def test_training_step_in_two_graphs(rows, given):
    """Two graphs of the same leaves, each with workspaces of its own, replayed in
    turn while an eager autograd graph of the leaves lives."""
    gu.say(f"graphs of the training step, {rows} rows")
    width, hidden = 512, 264
    g = gen(rows)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()   # noqa: E731
    gain, shift, wg, wu = (t.requires_grad_() for t in (r(width), r(width), r(hidden, width) / 16, r(hidden, width) / 16))
    xs, dys = [r(rows, width) for _ in range(2)], [r(rows, hidden) for _ in range(2)]
    alive = mxq.autograd.gated(mxq.autograd.layer_norm(xs[0].clone(), gain, shift), wg, wu)
    alive.sum().backward(retain_graph=True)
    spaces = [None, None]
    if given:
        sizes = (mxq.workspace_size(_lib.OP_GATED_BACKWARD, rows, hidden, width),
                 mxq.workspace_size(_lib.OP_LAYER_NORM_BACKWARD, rows, width))
        spaces = [tuple(torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes) for _ in range(2)]
    leaves = [t.detach() for t in (gain, shift, wg, wu)]
    graphs, outs = [], []
    for i in range(2):
        step(xs[i], dys[i], *leaves, spaces[i])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(xs[i], dys[i], *leaves, spaces[i]))
        graphs.append(graph)
    for rep in range(4):
        for i in range(2):
            xs[i].copy_(r(rows, width))
            dys[i].copy_(r(rows, hidden))
        want = [step(xs[i], dys[i], *leaves, None) for i in range(2)]
        for o in outs[0] + outs[1]:
            o.fill_(7)
        for i in (rep % 2, 1 - rep % 2):
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            for k, (a, b) in enumerate(zip(outs[i], want[i])):
                assert torch.equal(a, b), (rep, i, k)
    alive.sum().backward()


def test_two_streams_at_once():
    """The same operators on two streams, launched in turn without waits."""
    g = gen(21)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()   # noqa: E731
    args = [(r(300, 512), r(300, 264), r(512), r(512), r(264, 512) / 16, r(264, 512) / 16) for _ in range(2)]
    want = [step(*a, None) for a in args]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(step(*args[i], None))
    torch.cuda.synchronize()
    for i in range(2):
        for outs in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(outs, want[i]))


def _calls():
    x = torch.ones(8, 256, device="cuda")
    xb, w = x.bfloat16(), torch.ones(128, 256, dtype=BF, device="cuda")
    a, wt = mxq.quantize(x, mxq.FP8), mxq.quantize(w, mxq.FP8_TILE)
    off = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    perm = torch.arange(128, dtype=torch.int32, device="cuda")
    ops = [mxq.bf16_operand(t) for t in (xb, w, w)]
    saved, dy = torch.ones(2, 8, 128, device="cuda"), torch.ones(8, 128, dtype=BF, device="cuda")
    stats = torch.ones(8, 2, device="cuda")
    return {
        "quantize": lambda s: mxq.quantize(x, mxq.FP8, stream=s),
        "gemm": lambda s: mxq.gemm(a, wt, stream=s),
        "gemm_mixed": lambda s: mxq.gemm_mixed(a, [wt], perm, 128, stream=s),
        "gemm_grouped": lambda s: mxq.gemm_grouped(a, wt, off, stream=s),
        "gemm_gated": lambda s: mxq.gemm_gated(a, wt, wt, stream=s),
        "gemm_gated_backward": lambda s: mxq.gemm_gated_backward(dy, *ops, saved, stream=s),
        "layer_norm": lambda s: mxq.layer_norm(x, stream=s),
        "layer_norm_backward": lambda s: mxq.layer_norm_backward(x, x, stats, stream=s),
    }


@pytest.mark.parametrize("name", ["quantize", "gemm", "gemm_mixed", "gemm_grouped", "gemm_gated", "gemm_gated_backward",
                                  "layer_norm", "layer_norm_backward"])
def test_allocations_are_the_given_streams(name):
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
    parts = lambda t: (t.codes, t.scales) if isinstance(t, mxq.QTensor) else t if isinstance(t, tuple) else (t,)   # noqa: E731
    assert all(torch.equal(a, b) for a, b in zip(parts(got), parts(want)))


@pytest.mark.parametrize("fmt", [mxq.FP8, mxq.FP8_TILE])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nonfinite_input_flags_the_next_call(fmt, bad, monkeypatch):
    monkeypatch.setenv("MXQ_DEBUG_CHECKS", "1")
    x = torch.ones(9, 160, device="cuda")
    mxq.quantize(x, fmt)
    mxq.quantize(x, fmt)
    y = x.clone()
    y[7, 150] = bad
    mxq.quantize(y, fmt)
    with pytest.raises(_lib.MxqError) as e:
        mxq.layer_norm(x)
    assert e.value.status == 8
    mxq.quantize(x, fmt)


# ---- refusals of the binding ----------------------------------------------

def z(*size, dtype=F32, device="cuda"):
    return torch.zeros(size, dtype=dtype, device=device)


M, N, K = 6, 40, 64


@pytest.mark.parametrize("kw", [
    dict(out=z(M, N, device="cpu")), dict(out=z(M, N, dtype=BF, device="cpu")), dict(saved=z(2, M, N, device="cpu")),
], ids=["f32 host", "host", "saved host"])
def test_gated_refuses_host_outputs(kw):
    ops = [mxq.bf16_operand(z(r, K, dtype=BF)) for r in (M, N, N)]
    with pytest.raises(ValueError):
        mxq.gemm_gated(*ops, **kw)


def test_gated_refuses():
    ops = [mxq.bf16_operand(z(r, K, dtype=BF)) for r in (M, N, N)]
    for kw in (dict(out=z(M, N)), dict(out=z(M - 1, N, dtype=BF)), dict(out=z(N, M, dtype=BF).t()),
               dict(out=z(M, 2 * N, dtype=BF)[:, ::2]), dict(saved=z(2, M, N, dtype=BF)), dict(saved=z(2, M - 1, N)),
               dict(saved=z(2, M, N + 1)[:, :, :N]), dict(saved=z(M, N)), dict(out=z(M * N, dtype=BF))):
        with pytest.raises(ValueError):
            mxq.gemm_gated(*ops, **kw)
    with pytest.raises((ValueError, KeyError, _lib.MxqError)):
        mxq.gemm_gated(*ops, act="relu")
    with pytest.raises(_lib.MxqError):
        mxq.gemm_gated(ops[0], ops[1], mxq.bf16_operand(z(N - 1, K, dtype=BF)))
    q = mxq.quantize(z(M, K), mxq.FP8)
    with pytest.raises(_lib.MxqError):
        mxq.gemm_gated(q, *ops[1:])
    dy, saved = z(M, N, dtype=BF), z(2, M, N)
    for a, kw in (((z(M, N), saved), {}), ((z(M - 1, N, dtype=BF), saved), {}), ((z(N, M, dtype=BF).t(), saved), {}),
                  ((dy, z(2, M, N - 1)), {}), ((dy, z(2, M, N, dtype=BF)), {}), ((dy, saved), dict(dx=z(M, K))),
                  ((dy, saved), dict(dx=z(M, K - 1, dtype=BF))), ((dy, saved), dict(dw_gate=z(N, K), dw_up=z(N, K, dtype=BF))),
                  ((dy, saved), dict(dw_gate=z(N, K + 8, dtype=BF)[:, :K])),
                  ((dy, saved), dict(workspace=z(2, 1 << 20, dtype=torch.uint8)[:, ::2]))):
        with pytest.raises(ValueError):
            mxq.gemm_gated_backward(a[0], *ops, a[1], **kw)
    with pytest.raises(_lib.MxqError):
        mxq.gemm_gated_backward(dy, *ops, saved, workspace=z(16, dtype=torch.uint8))


def test_layer_norm_refuses():
    x, st = z(5, 24, dtype=BF), z(5, 2)
    for a, kw in (((z(5, 24, dtype=torch.float16),), {}), ((z(5, 24, dtype=torch.float64),), {}), ((z(24, dtype=BF),), {}),
                  ((z(24, 5, dtype=BF).t(),), {}), ((x, z(24)), {}), ((x, z(23, dtype=BF)), {}), ((x, z(48, dtype=BF)[::2]), {}),
                  ((x, None, z(24)), {}), ((x,), dict(out=z(5, 24))), ((x,), dict(out=z(4, 24, dtype=BF))),
                  ((x,), dict(stats=z(5, 2, dtype=BF))), ((x,), dict(stats=z(4, 2))), ((x,), dict(stats=z(5, 3)[:, :2])),
                  ((x,), dict(stats=z(5, 2, device="cpu")))):
        with pytest.raises(ValueError):
            mxq.layer_norm(*a, **kw)
    with pytest.raises(_lib.MxqError):
        mxq.layer_norm(x, eps=-1e-5)
    for a, kw in (((z(5, 24), x, st), {}), ((x[:4], x, st), {}), ((x, x, z(5, 2, dtype=BF)), {}), ((x, x, st, z(24)), {}),
                  ((x, x, st), dict(dx=z(5, 24))), ((x, x, st), dict(dweight=z(24))), ((x, x, st), dict(dbias=z(25, dtype=BF))),
                  ((x, x, st), dict(workspace=z(2, 1 << 20, dtype=torch.uint8)[:, ::2]))):
        with pytest.raises(ValueError):
            mxq.layer_norm_backward(*a, **kw)
    with pytest.raises(_lib.MxqError):
        mxq.layer_norm_backward(x, x, st, workspace=z(16, dtype=torch.uint8))


# ---- offsets that pass 32 bits ---------------------------------------------

def test_rows_far_apart():
    """Rows 2**31 + 8 elements apart."""
    gu.say("layer norm and quantize, rows 2**31 apart")
    ld = (1 << 31) + 8
    base = torch.empty(2 * ld + 256, dtype=BF, device="cuda")
    x = base.as_strided((3, 256), (ld, 1))
    x.copy_(torch.randn((3, 256), generator=gen(1), device="cuda"))
    near, dy = x.contiguous(), torch.randn((3, 256), generator=gen(2), device="cuda").bfloat16()
    st = [torch.empty((3, 2), device="cuda") for _ in range(2)]
    assert torch.equal(mxq.layer_norm(x, stats=st[0]), mxq.layer_norm(near, stats=st[1])) and torch.equal(*st)
    for a, b in zip(mxq.layer_norm_backward(dy, x, st[0]), mxq.layer_norm_backward(dy, near, st[0])):
        assert torch.equal(a, b)
    for fmt in (mxq.FP8, mxq.FP8_TILE):
        a, b = mxq.quantize(x, fmt), mxq.quantize(near, fmt)
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    want = mxq.layer_norm(near)
    mxq.layer_norm(x, out=x)
    assert torch.equal(x, want)


def test_more_than_2_to_31_outputs():
    """Pre-activations, outputs and gradients of 70001 x 33000, exact sums, looked at
    in rows and columns of the first and last tiles."""
    gu.say("gated 70001x33000x8, exact sums")
    m, n, k = 70001, 33000, 8
    g = gen(0)
    sign = lambda *s: (torch.randint(0, 2, s, generator=g, device="cuda").float() * 2 - 1).bfloat16()   # noqa: E731
    x, wg, wu = sign(m, k), sign(n, k), sign(n, k)
    x[:, 0], wg[:, 0], wu[:, 0] = 1, 128, 0
    dy = sign(m, n)
    ops = [mxq.bf16_operand(t) for t in (x, wg, wu)]
    saved = torch.empty((2, m, n), device="cuda")
    y = mxq.gemm_gated(*ops, saved=saved)
    dx, dwg, dwu = mxq.gemm_gated_backward(dy, *ops, saved)
    xd, gd, ud = x.double(), wg.double(), wu.double()
    for rows in (slice(0, 300), slice(65000, 65300), slice(m - 300, m)):
        gate, up = xd[rows] @ gd.t(), xd[rows] @ ud.t()
        assert torch.equal(saved[0, rows].double(), gate) and torch.equal(saved[1, rows].double(), up)
        assert torch.equal(y[rows], bf16(gate * up))
        dg, du = dy[rows].double() * up, dy[rows].double() * gate
        assert torch.equal(dx[rows], bf16(dg @ gd + du @ ud))
    for cols in (slice(0, 100), slice(n - 100, n)):
        gate, up = xd @ gd[cols].t(), xd @ ud[cols].t()
        d = dy[:, cols].double()
        assert torch.equal(dwg[cols], bf16((d * up).t() @ xd)) and torch.equal(dwu[cols], bf16((d * gate).t() @ xd))


@pytest.mark.parametrize("m,n,k", [(3, 130, 65600), (200, 264, 40000)])
def test_long_sums(m, n, k):
    gu.say(f"gated {m}x{n}x{k} bf16, exact sums")
    x, wg, wu, dy, gate, up = exact_case(m, n, k)
    ops = [mxq.bf16_operand(t.bfloat16()) for t in (x, wg, wu)]
    saved = torch.empty((2, m, n), device="cuda")
    assert torch.equal(mxq.gemm_gated(*ops, saved=saved), bf16(gate * up))
    got = mxq.gemm_gated_backward(dy.bfloat16(), *ops, saved)
    dg, du = dy.double() * up, dy.double() * gate
    for a, b in zip(got, (dg @ wg.double() + du @ wu.double(), dg.t() @ x.double(), du.t() @ x.double())):
        assert torch.equal(a, bf16(b))
