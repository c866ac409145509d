"""The layer norm where its loops and its shapes repeat: several rows to a group of
waves in every shape of the gradients, rows too long for the registers at any
alignment, strides and results in place at each width.  Against float64."""
import pytest
import torch

import fp8_quantized_linear_mxq_amd as mxq
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def draw(rows, cols, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")   # noqa: E731
    x = (r(rows, cols) * torch.exp(r(cols)) + 0.5).to(DT[dtype])
    return x, (1 + 0.2 * r(cols)).to(DT[dtype]), (0.3 * r(cols)).to(DT[dtype]), r(rows, cols).to(DT[dtype])


def half(dtype):
    return 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24


def within(got, want, tol, what):
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), f"{what}: worst {float((err / tol).max()):.3g} of the bound"


class Exact:
    """The formulas in float64, and what their fp32 evaluation may be off by.

    u: roundings that a sum over a row passes, of its absolute terms.  A lane adds at
    most 64 elements in registers, in the shapes that read a row several times
    (256 lanes and more) cols / 256 and a piece of eight; then six joins of lanes
    and sixteen of waves.  v: the same over rows.  256 workgroups take rows / 256 and one
    more between them, at worst all by one thread; then sixteen groups of waves in
    LDS, sixteen workgroups' shares to a wave, sixteen waves."""

    def __init__(self, x, w, b, dy, dtype):
        rows, cols = x.shape
        self.dtype = dtype
        x, w, b, dy = (t.double() for t in (x, w, b, dy))
        u = (max(64, cols / 256 + 8) + 6 + 16) * 2.0 ** -24
        v = (rows / 256 + 1 + 16 + 16 + 16) * 2.0 ** -24
        row = lambda t: t.mean(dim=1, keepdim=True)   # noqa: E731
        self.mean = row(x)
        d = x - self.mean
        self.rstd = 1 / (row(d * d) + EPS).sqrt()
        h = d * self.rstd
        self.y = h * w + b
        # the mean's error, and that of the mean square through h; a few roundings on the way
        self.emean = u * row(x.abs())
        eh = self.rstd * self.emean * (1 + h.abs()) + h.abs() * (u + 2.0 ** -20) + self.rstd * x.abs() * 2.0 ** -24
        self.ty = eh * w.abs() + b.abs() * 2.0 ** -23 + (half(dtype) + 2.0 ** -23) * self.y.abs() + 2.0 ** -133
        t = dy * w
        m1, m2 = row(t.abs()), row((t * h).abs())
        self.dx = self.rstd * (t - row(t) - h * row(t * h))
        e = self.rstd * ((u + 2.0 ** -20) * (t.abs() + m1 + h.abs() * m2) + eh * m2 + h.abs() * row(t.abs() * eh))
        self.tx = e + (u + 2.0 ** -20 + half(dtype)) * self.dx.abs() + 2.0 ** -133
        self.dw, self.db = (dy * h).sum(dim=0), dy.sum(dim=0)
        self.tw = (v + 2.0 ** -22) * (dy * h).abs().sum(dim=0) + (dy.abs() * eh).sum(dim=0) + \
            half(dtype) * self.dw.abs() + 2.0 ** -133
        self.tb = v * dy.abs().sum(dim=0) + half(dtype) * self.db.abs() + 2.0 ** -133

    def forward(self, y, stats):
        within(y, self.y, self.ty, "y")
        within(stats[:, :1], self.mean, self.emean + 1e-30, "mean")

    def gradients(self, got):
        for name, g in zip(("dx", "dw", "db"), got):
            within(g, getattr(self, name), getattr(self, "t" + name[1]), name)


# three rows and more to each group of waves of each shape: rows > 2 * 256 * (groups in a workgroup)
SHAPES = [(8300, 264), (8300, 1024), (5000, 1536), (2100, 4096), (1100, 8192), (600, 16384),   # whole, aligned pieces
          (600, 16400),                                                                        # too long for registers
          (8300, 63), (8300, 257), (4200, 1001),                                               # single elements
          (4200, 1030), (2100, 4090), (1100, 8001), (600, 12345),                              # pieces at any alignment
          (600, 16401), (7, 16385), (7, 20001)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_several_rows_to_a_group(rows, cols, dtype):
    gu.say(f"layer norm {rows}x{cols} {dtype}")
    x, w, b, dy = draw(rows, cols, dtype, rows + cols)
    want = Exact(x, w, b, dy, dtype)
    stats = torch.empty((rows, 2), device="cuda")
    want.forward(mxq.layer_norm(x, w, b, stats=stats), stats)
    got = mxq.layer_norm_backward(dy, x, stats, w)
    want.gradients(got)
    again = mxq.layer_norm_backward(dy, x, stats, w)
    assert all(torch.equal(p, q) for p, q in zip(got, again))
    only = mxq.layer_norm_backward(dy, x, stats, w, want=(False, True))
    assert torch.equal(only[1], got[1]) and torch.equal(only[2], got[2])


@pytest.mark.parametrize("cols", [264, 2048, 4090, 16392])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_alignment_and_in_place(cols, dtype):
    """Rows of wider tensors at every alignment of their first element: values, gaps
    that keep theirs, results in place of x and of dy."""
    rows = 33
    gu.say(f"layer norm {rows}x{cols} {dtype}, strides")
    x, w, b, dy = draw(rows, cols, dtype, cols)
    want = Exact(x, w, b, dy, dtype)

    def part(first, width, t, gap):
        wide = torch.full((rows, width), gap, dtype=DT[dtype], device="cuda")
        wide[:, first:first + cols] = t
        return wide, wide[:, first:first + cols]

    for first, width in ((0, cols), (8, cols + 24), (1, cols + 1), (3, cols + 7), (2, cols + 8)):
        xs, ds = part(first, width, x, float("nan"))[1], part(first, width, dy, float("nan"))[1]
        ys, y = part(first, width, x.new_full((rows, cols), 5.0), -7.0)
        gs, dx = part(first, width, x.new_full((rows, cols), 5.0), -7.0)
        stats = torch.empty((rows, 2), device="cuda")
        mxq.layer_norm(xs, w, b, out=y, stats=stats)
        want.forward(y, stats)
        grads = mxq.layer_norm_backward(ds, xs, stats, w, dx=dx)
        want.gradients(grads)
        for t in (ys, gs):
            assert bool((t[:, :first] == -7).all()) and bool((t[:, first + cols:] == -7).all())
        wx, px = part(first, width, x, -7.0)
        assert mxq.layer_norm(px, w, b, out=px) is px and torch.equal(px, y)
        assert bool((wx[:, :first] == -7).all()) and bool((wx[:, first + cols:] == -7).all())
        for into in (0, 1):
            pair = [part(first, width, t, -7.0) for t in (dy, x)]
            got = mxq.layer_norm_backward(pair[0][1], pair[1][1], stats, w, dx=pair[into][1])
            assert all(torch.equal(p, q) for p, q in zip(got, grads))
            assert bool((pair[into][0][:, :first] == -7).all()) and bool((pair[into][0][:, first + cols:] == -7).all())
