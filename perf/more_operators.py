"""Timed cases of the 8-bit floating point layer, the gated feed-forward and the layer norm.

Four operators, each in a plain form (elementary torch operations in float32, in
float64 next to a rounding border, rounded once at the end) and, with ``own`` set,
through this package's entry points:

  quantize  E4M3 codes with one float32 scale per row and 128 columns (activations)
            or per 128 x 128 tile (weights)
  gemm      product of such activations and weights, with a bias
  gated     act(x Wg^T) * (x Wu^T): on the 8-bit operands for serving; in bfloat16,
            alone or as a training step with the gradients of x, Wg and Wu
  norm      layer norm, alone or with the gradients of x, the weight and the bias
"""
import math

import torch

own = False


def listed():
    return [
        # a decode batch of 37 sequences entering a 1184-wide layer: latency, a last block of 32
        {"name": "quantize_batch", "op": "quantize", "m": 37, "k": 1184, "dtype": "bf16", "tile": False},
        # a long batch of 4608-wide MLP activations: memory traffic
        {"name": "quantize_long", "op": "quantize", "m": 16384, "k": 4608, "dtype": "bf16", "tile": False},
        # one token through a wide projection: weight traffic and latency
        {"name": "gemm_token", "op": "gemm", "m": 1, "k": 4096, "n": 8192, "bias": True},
        # an odd batch through a projection of odd width
        {"name": "gemm_ragged", "op": "gemm", "m": 777, "k": 1184, "n": 1001, "bias": False},
        # a large square layer: matrix-core throughput
        {"name": "gemm_large", "op": "gemm", "m": 8192, "k": 8192, "n": 8192, "bias": False},
        # one token through both projections of a feed-forward block on 8-bit weights
        {"name": "gated_token", "op": "gated", "kind": "fp8", "m": 1, "k": 4096, "n": 11008, "act": "silu"},
        # a 4096-token prompt through the same block
        {"name": "gated_prompt", "op": "gated", "kind": "fp8", "m": 4096, "k": 4096, "n": 11008, "act": "silu"},
        # a training step on a short batch of odd sizes
        {"name": "gated_train_ragged", "op": "gated", "kind": "train", "m": 1111, "k": 1160, "n": 2003, "act": "gelu"},
        # a training step on 8192 tokens
        {"name": "gated_train", "op": "gated", "kind": "train", "m": 8192, "k": 2048, "n": 5632, "act": "silu"},
        # one token of a 1152-wide layer: launch latency is all there is
        {"name": "norm_token", "op": "norm", "m": 1, "k": 1152, "dtype": "bf16", "train": False},
        # a long batch in front of a 4096-wide layer: memory traffic
        {"name": "norm_long", "op": "norm", "m": 16384, "k": 4096, "dtype": "bf16", "train": False},
        # a training step's norm, forward and backward
        {"name": "norm_train", "op": "norm", "m": 8192, "k": 4096, "dtype": "bf16", "train": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "gemm", "gemm", "gated", "gated", "gated", "norm", "norm"))
    if op == "quantize":
        return {"op": op, "m": _log(rng, 1, 16384), "k": 32 * _log(rng, 2, 144),
                "dtype": rng.choice(("bf16", "bf16", "f32")), "tile": rng.random() < 0.3}
    if op == "gemm":
        return {"op": op, "m": _log(rng, 1, 8192), "k": 32 * _log(rng, 8, 256),
                "n": _log(rng, 64, 8192), "bias": rng.random() < 0.5}
    if op == "gated":
        kind = rng.choice(("fp8", "bf16", "train"))
        unit = 32 if kind == "fp8" else 8
        return {"op": op, "kind": kind, "m": _log(rng, 1, 4096), "k": unit * _log(rng, 256 // unit, 4096 // unit),
                "n": _log(rng, 64, 5632), "act": rng.choice(("silu", "gelu", "gelu_tanh"))}
    return {"op": op, "m": _log(rng, 1, 8192), "k": _log(rng, 32, 4096),
            "dtype": rng.choice(("bf16", "bf16", "f32")), "train": rng.random() < 0.6}


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _heavy(g, m, k):
    """Activations: normal with a few strong channels, as after a norm."""
    x = torch.randn((m, k), generator=g, device="cuda")
    return x * torch.exp(torch.randn((k,), generator=g, device="cuda"))


def _blocks(x, rows):
    """x [m, k] as [m / rows, rows, k / 128, 128], padded with zeros."""
    m, k = x.shape
    x = torch.nn.functional.pad(x, (0, -k % 128, 0, -m % rows))
    return x.view(-1, rows, x.shape[1] // 128, 128)


def _spread(s, rows, m, k):
    """Scales per block [m / rows, k / 128] to every element [m, k]."""
    return s.repeat_interleave(rows, 0)[:m].repeat_interleave(128, 1)[:, :k]


def _codes(x, rows):
    """E4M3 codes and scales of inputs that are already quantized."""
    s = _blocks(x, rows).abs().amax(dim=(1, 3)) / 448.0
    q = (x / _spread(s, rows, *x.shape)).clamp(-448, 448)
    return q.to(torch.float8_e4m3fn), s


def prepare(case, seed):
    g = _generator(seed)
    m, k = case["m"], case["k"]
    st = {"case": case}
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    if case["op"] == "quantize":
        x = 0.02 * randn(m, k) if case["tile"] else _heavy(g, m, k)
        st["x"] = x.to(_dtype(case["dtype"]))
    elif case["op"] == "gemm" or case.get("kind") == "fp8":
        a, sa = _codes(_heavy(g, m, k), 1)
        st["a"], st["sa"] = a, sa.t().contiguous()      # scales: the rows of a block of columns lie together
        for name in ("w",) if case["op"] == "gemm" else ("wg", "wu"):
            st[name], st["s" + name] = _codes(k ** -0.5 * randn(case["n"], k), 128)
        if case.get("bias"):
            st["bias"] = randn(case["n"]).to(torch.bfloat16)
    elif case["op"] == "gated":
        st["x"] = randn(m, k).to(torch.bfloat16)
        st["wg"] = (k ** -0.5 * randn(case["n"], k)).to(torch.bfloat16)
        st["wu"] = (k ** -0.5 * randn(case["n"], k)).to(torch.bfloat16)
        if case["kind"] == "train":
            st["dy"] = randn(m, case["n"]).to(torch.bfloat16)
    else:
        dt = _dtype(case["dtype"])
        st["x"] = (_heavy(g, m, k) + randn(m, 1)).to(dt)
        st["w"] = (1 + 0.1 * randn(k)).to(dt)
        st["b"] = (0.1 * randn(k)).to(dt)
        if case["train"]:
            st["dy"] = randn(m, k).to(dt)
    return st


def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


# ---- plain forms ----------------------------------------------------------

def _plain_quantize(st):
    rows = 128 if st["case"]["tile"] else 1
    x = st["x"].double()     # the quotient's side of a rounding border, exactly
    s = (_blocks(x, rows).abs().amax(dim=(1, 3)) / 448.0).float()
    d = _spread(s, rows, *x.shape).double()
    v = torch.where(d > 0, x / d, torch.zeros_like(x)).clamp(-448, 448)
    # E4M3: eight steps to a binade, 2**-9 at least
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    q = (torch.round(v / step) * step).float()
    return {"codes": q.to(torch.float8_e4m3fn), "scales": s if st["case"]["tile"] else s.t().contiguous()}


def _values(codes, scales, rows):
    return codes.float() * _spread(scales, rows, *codes.shape)


def _plain_gemm(st):
    y = _values(st["a"], st["sa"].t(), 1) @ _values(st["w"], st["sw"], 128).t()
    if "bias" in st:
        y = y + st["bias"].float()
    return y.to(torch.bfloat16)


def _act(g, name):
    """The activation and its derivative."""
    if name == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    if name == "gelu":
        c = 0.5 * torch.erfc(-g * 0.5 ** 0.5)
        return g * c, c + g * torch.exp(-0.5 * g * g) * (2 * math.pi) ** -0.5
    a = (2 / math.pi) ** 0.5
    s = 1 / (1 + torch.exp(-2 * a * (g + 0.044715 * g * g * g)))   # (1 + tanh) / 2
    return g * s, s + 2 * a * g * (1 + 3 * 0.044715 * g * g) * s * (1 - s)


def _plain_gated(st):
    c = st["case"]
    if c["kind"] == "fp8":
        x = _values(st["a"], st["sa"].t(), 1)
        wg, wu = _values(st["wg"], st["swg"], 128), _values(st["wu"], st["swu"], 128)
    else:
        x, wg, wu = st["x"].float(), st["wg"].float(), st["wu"].float()
    g, u = x @ wg.t(), x @ wu.t()
    f, df = _act(g, c["act"])
    y = (f * u).to(torch.bfloat16)
    if c["kind"] != "train":
        return y
    dy = st["dy"].float()
    dg, du = dy * u * df, dy * f
    return {"y": y, "dx": (dg @ wg + du @ wu).to(torch.bfloat16),
            "dwg": (dg.t() @ x).to(torch.bfloat16), "dwu": (du.t() @ x).to(torch.bfloat16)}


def _plain_norm(st):
    x, w = st["x"].float(), st["w"].float()
    dt = st["x"].dtype
    x = x - x.mean(dim=1, keepdim=True)
    rstd = torch.rsqrt((x * x).mean(dim=1, keepdim=True) + 1e-5)
    xh = x * rstd
    y = (xh * w + st["b"].float()).to(dt)
    if not st["case"]["train"]:
        return y
    dy = st["dy"].float()
    t = dy * w
    dx = rstd * (t - t.mean(dim=1, keepdim=True) - xh * (t * xh).mean(dim=1, keepdim=True))
    return {"y": y, "dx": dx.to(dt), "dw": (dy * xh).sum(dim=0).to(dt), "db": dy.sum(dim=0).to(dt)}


_plain = {"quantize": _plain_quantize, "gemm": _plain_gemm, "gated": _plain_gated, "norm": _plain_norm}


# ---- through the package --------------------------------------------------

def _own_quantize(st):
    import fp8_quantized_linear_mxq_amd as mxq
    q = mxq.quantize(st["x"], mxq.FP8_TILE if st["case"]["tile"] else mxq.FP8)
    return {"codes": q.codes[:, :q.cols].view(torch.float8_e4m3fn), "scales": q.scales}


def _own_gemm(st):
    import fp8_quantized_linear_mxq_amd as mxq
    return mxq.gemm(mxq.fp8_operand(st["a"], st["sa"]), mxq.fp8_operand(st["w"], st["sw"], tile=True),
                    bias=st.get("bias"))


def _own_gated(st):
    import fp8_quantized_linear_mxq_amd as mxq
    c = st["case"]
    if c["kind"] == "fp8":
        return mxq.gemm_gated(mxq.fp8_operand(st["a"], st["sa"]), mxq.fp8_operand(st["wg"], st["swg"], tile=True),
                              mxq.fp8_operand(st["wu"], st["swu"], tile=True), act=c["act"])
    x, wg, wu = (mxq.bf16_operand(st[n]) for n in ("x", "wg", "wu"))
    if c["kind"] == "bf16":
        return mxq.gemm_gated(x, wg, wu, act=c["act"])
    saved = torch.empty((2, c["m"], c["n"]), dtype=torch.float32, device="cuda")
    y = mxq.gemm_gated(x, wg, wu, act=c["act"], saved=saved)
    dx, dwg, dwu = mxq.gemm_gated_backward(st["dy"], x, wg, wu, saved, act=c["act"])
    return {"y": y, "dx": dx, "dwg": dwg, "dwu": dwu}


def _own_norm(st):
    import fp8_quantized_linear_mxq_amd as mxq
    if not st["case"]["train"]:
        return mxq.layer_norm(st["x"], st["w"], st["b"], eps=1e-5)
    stats = torch.empty((st["case"]["m"], 2), dtype=torch.float32, device="cuda")
    y = mxq.layer_norm(st["x"], st["w"], st["b"], eps=1e-5, stats=stats)
    dx, dw, db = mxq.layer_norm_backward(st["dy"], st["x"], stats, st["w"])
    return {"y": y, "dx": dx, "dw": dw, "db": db}


_own = {"quantize": _own_quantize, "gemm": _own_gemm, "gated": _own_gated, "norm": _own_norm}


# ---- what cannot be avoided, and the values in 64 bits --------------------

def work(case):
    m, k = case["m"], case["k"]
    kb = -(-k // 128)
    if case["op"] == "quantize":
        scales = 4 * kb * (-(-m // 128) if case["tile"] else m)
        return {"bytes": m * k * ((2 if case["dtype"] == "bf16" else 4) + 1) + scales, "flops": 4 * m * k}
    if case["op"] == "norm":
        size, n = 2 if case["dtype"] == "bf16" else 4, m * k * (4 if case["train"] else 2)
        return {"bytes": size * (n + (5 if case["train"] else 2) * k), "flops": (18 if case["train"] else 8) * m * k}
    n = case["n"]
    tiles = 4 * kb * (m + -(-n // 128))      # scales
    if case["op"] == "gemm":
        return {"bytes": m * k + n * k + tiles + 2 * m * n + (2 * n if case["bias"] else 0), "flops": 2 * m * n * k}
    if case["kind"] == "fp8":
        return {"bytes": m * k + 2 * n * k + 4 * kb * (m + 2 * -(-n // 128)) + 2 * m * n, "flops": 4 * m * n * k}
    if case["kind"] == "bf16":
        return {"bytes": 2 * (m * k + 2 * n * k + m * n), "flops": 4 * m * n * k}
    return {"bytes": 2 * (2 * m * k + 4 * n * k + 2 * m * n), "flops": 12 * m * n * k}


def _pow2(e):
    """2**e of whole numbers in [-32, 32], from a table: a device pow may be a rounding off."""
    return torch.tensor([2.0 ** i for i in range(-32, 33)], dtype=torch.float64, device=e.device)[e.long() + 32]


def _exact_values(codes, scales, rows):
    """Every element from its bits, times its block's scale."""
    c = codes.view(torch.uint8).long()
    e, f = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e > 0, (1 + f / 8) * _pow2(e - 7), f * 2.0 ** -9)
    v = torch.where(c >= 128, -v, v)
    r = torch.arange(v.shape[0], device=v.device) // rows
    col = torch.arange(v.shape[1], device=v.device) // 128
    return v * scales.double()[r][:, col]


def _exact_gate(g, name):
    """Activation and derivative, the derivative by its own formula."""
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * torch.sigmoid(-g)
    if name == "gelu":
        c = torch.special.ndtr(g)
        return g * c, c + g * torch.exp(-g.square() / 2) / math.sqrt(2 * math.pi)
    z = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    t = torch.tanh(z)
    return g * (1 + t) / 2, (1 + t) / 2 + g / 2 * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 0.134145 * g.square())


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        rows = 128 if case["tile"] else 1
        x = st["x"].double()
        m, k = x.shape
        kb = -(-k // 128)
        s = torch.zeros((-(-m // rows), kb), dtype=torch.float64, device="cuda")
        for j in range(kb):      # each block of columns by itself
            top = x[:, 128 * j:128 * j + 128].abs().max(dim=1).values
            s[:, j] = torch.stack([p.max() for p in top.split(rows)]) if case["tile"] else top
        s = (s / 448).float().double()
        d = s[torch.arange(m, device="cuda") // rows][:, torch.arange(k, device="cuda") // 128]
        v = (x / torch.where(d == 0, torch.ones_like(d), d)).clamp(-448, 448)
        e = (torch.frexp(v).exponent - 1).clamp_min(-6)       # v = f 2**(e + 1), 1/2 <= |f| < 1
        q = (v * _pow2(3 - e)).round() * _pow2(e - 3)
        return {"codes": q, "scales": s if case["tile"] else s.T.contiguous()}
    if op == "gemm":
        y = _exact_values(st["a"], st["sa"].T, 1) @ _exact_values(st["w"], st["sw"], 128).T
        return y + st["bias"].double() if "bias" in st else y
    if op == "gated":
        if case["kind"] == "fp8":
            x = _exact_values(st["a"], st["sa"].T, 1)
            wg, wu = _exact_values(st["wg"], st["swg"], 128), _exact_values(st["wu"], st["swu"], 128)
        else:
            x, wg, wu = st["x"].double(), st["wg"].double(), st["wu"].double()
        g, u = x @ wg.T, x @ wu.T
        f, df = _exact_gate(g, case["act"])
        if case["kind"] != "train":
            return f * u
        dy = st["dy"].double()
        dg, du = dy * u * df, dy * f
        return {"y": f * u, "dx": dg @ wg + du @ wu, "dwg": dg.T @ x, "dwu": du.T @ x}
    x, w, k = st["x"].double(), st["w"].double(), case["k"]
    mean = x.sum(dim=1, keepdim=True) / k
    std = ((x - mean).square().sum(dim=1, keepdim=True) / k + 1e-5).sqrt()
    xh = (x - mean) / std
    y = xh * w + st["b"].double()
    if not case["train"]:
        return y
    dy = st["dy"].double()
    t = dy * w
    dx = (t - (t.sum(dim=1, keepdim=True) + xh * (t * xh).sum(dim=1, keepdim=True)) / k) / std
    return {"y": y, "dx": dx, "dw": torch.einsum("ij,ij->j", dy, xh), "db": dy.sum(dim=0)}
