"""Timed cases of the int8, expert-grouped and head-norm operators.

Four operators, each in a plain form (elementary torch operations in float32,
rounded once at the end) and, with ``own`` set, through this package's entry
points:

  quantize  row-wise int8 quantization of activations
  gemm      int8 x int8 product with a scale per token and per output channel
  grouped   products grouped by expert, group sizes on the device
            (int8 x int8, MXFP4 x MXFP4, bf16 x MXFP4)
  qknorm    RMS norm of every query and key head with the position rotation
"""
import math

import torch

own = False

# E2M1 magnitudes by code, then the negative half
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token entering a 1152-wide layer: launch latency is all there is
        {"name": "quantize_token", "op": "quantize", "m": 1, "k": 1152, "dtype": "bf16"},
        # a long batch of 4608-wide MLP activations: memory traffic
        {"name": "quantize_long", "op": "quantize", "m": 16384, "k": 4608, "dtype": "bf16"},
        # one token through the MLP up-projection: weight traffic and latency
        {"name": "gemm_token", "op": "gemm", "m": 1, "k": 1152, "n": 4608, "bias": True},
        # an odd batch through a projection of odd width
        {"name": "gemm_ragged", "op": "gemm", "m": 777, "k": 1184, "n": 1001, "bias": False},
        # the MLP up-projection on 4096 tokens
        {"name": "gemm_mlp", "op": "gemm", "m": 4096, "k": 1152, "n": 4608, "bias": True},
        # a large square layer: matrix-core throughput
        {"name": "gemm_large", "op": "gemm", "m": 8192, "k": 8192, "n": 8192, "bias": False},
        # one token routed to 8 of 64 experts
        {"name": "grouped_i8_token", "op": "grouped", "pair": "i8", "tokens": 1, "topk": 8,
         "experts": 64, "k": 2048, "n": 1536},
        # a 2048-token prompt, 8 of 64 experts each
        {"name": "grouped_i8_prompt", "op": "grouped", "pair": "i8", "tokens": 2048, "topk": 8,
         "experts": 64, "k": 2048, "n": 1536},
        # a decode batch of 16 sequences, 4-bit weights and 16-bit activations
        {"name": "grouped_w4a16_batch", "op": "grouped", "pair": "w4a16", "tokens": 16, "topk": 4,
         "experts": 32, "k": 4096, "n": 2048},
        # a 4096-token prompt on 4-bit weights and activations
        {"name": "grouped_mx4_prompt", "op": "grouped", "pair": "mx4", "tokens": 4096, "topk": 4,
         "experts": 32, "k": 4096, "n": 2048},
        # one token of a 16 x 72 head layer (1152 wide)
        {"name": "qknorm_token", "op": "qknorm", "tokens": 1, "hq": 16, "hk": 16, "d": 72, "rot": 72,
         "pairs": "half", "dtype": "bf16"},
        # a long sequence with shared key heads
        {"name": "qknorm_long", "op": "qknorm", "tokens": 16384, "hq": 32, "hk": 8, "d": 128,
         "rot": 128, "pairs": "interleaved", "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "gemm", "gemm", "grouped", "grouped", "qknorm"))
    if op == "quantize":
        return {"op": op, "m": _log(rng, 1, 16384), "k": 32 * _log(rng, 2, 144),
                "dtype": rng.choice(("bf16", "bf16", "f32"))}
    if op == "gemm":
        return {"op": op, "m": _log(rng, 1, 8192), "k": 32 * _log(rng, 8, 256),
                "n": _log(rng, 64, 8192), "bias": rng.random() < 0.5}
    if op == "grouped":
        pair = rng.choice(("i8", "mx4", "w4a16"))
        unit = 32 if pair == "i8" else 128
        return {"op": op, "pair": pair, "tokens": _log(rng, 1, 2048 if pair == "w4a16" else 4096),
                "topk": rng.choice((1, 2, 4)), "experts": rng.choice((4, 16, 31, 32)),
                "k": unit * _log(rng, 512 // unit, 4096 // unit), "n": _log(rng, 256, 2048)}
    d = rng.choice((64, 72, 96, 128, 256))
    return {"op": op, "tokens": _log(rng, 1, 16384 * 40 * 128 // (24 * 256)), "hq": rng.choice((8, 15, 16)),
            "hk": rng.choice((1, 4, 8)), "d": d, "rot": rng.choice((d, d, d - 32)),
            "pairs": rng.choice(("half", "interleaved")), "dtype": rng.choice(("bf16", "bf16", "f32"))}


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _heavy(g, m, k):
    """Activations: normal with a few strong channels, as after a norm."""
    x = torch.randn((m, k), generator=g, device="cuda")
    spread = torch.exp(torch.randn((k,), generator=g, device="cuda"))
    return x * spread


def _int8(x):
    """Symmetric int8 codes and one scale per row, for inputs that are already quantized."""
    s = x.abs().amax(dim=1) / 127.0
    q = torch.round(x / s[:, None]).clamp(-127, 127).to(torch.int8)
    return q, s


def _mxfp4(x):
    """MXFP4 codes [rows, k/2] (low nibble first) and E8M0 scale codes [rows, k/32]."""
    rows, k = x.shape
    b = x.view(rows, k // 32, 32)
    e = torch.floor(torch.log2(b.abs().amax(dim=2).clamp_min(2.0 ** -100))) - 2
    v = b / torch.exp2(e)[:, :, None]
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    c = torch.bucketize(v.abs(), mids).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
    c = c.view(rows, k)
    return c[:, 0::2] | (c[:, 1::2] << 4), (e + 127).to(torch.uint8)


def _weights(make, g, experts, n, k):
    """One expert's weights at a time, so that the float32 draw stays small."""
    parts = [make(0.02 * torch.randn((n, k), generator=g, device="cuda")) for _ in range(experts)]
    return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    st = {"case": case}
    if op == "quantize":
        st["x"] = _heavy(g, case["m"], case["k"]).to(_dtype(case["dtype"]))
    elif op == "gemm":
        st["a"], st["sa"] = _int8(_heavy(g, case["m"], case["k"]))
        st["w"], st["sw"] = _weights(_int8, g, 1, case["n"], case["k"])
        st["bias"] = (torch.randn((case["n"],), generator=g, device="cuda").to(torch.bfloat16)
                      if case["bias"] else None)
    elif op == "grouped":
        t, e = case["tokens"], case["experts"]
        # a router with unequal experts: topk of noisy scores, rows sorted by expert
        liked = 0.5 * torch.randn((e,), generator=g, device="cuda")
        noise = torch.rand((t, e), generator=g, device="cuda").clamp_min(1e-9)
        picks = torch.topk(liked - torch.log(-torch.log(noise)), min(case["topk"], e), dim=1).indices
        counts = torch.bincount(picks.reshape(-1), minlength=e)
        st["cap"] = int(counts.max())
        st["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        x = _heavy(g, picks.numel(), case["k"])
        if case["pair"] == "i8":
            st["a"], st["sa"] = _int8(x)
        elif case["pair"] == "mx4":
            st["a"], st["sa"] = _mxfp4(x)
        else:
            st["a"], st["sa"] = x.to(torch.bfloat16), None
        st["w"], st["sw"] = _weights(_int8 if case["pair"] == "i8" else _mxfp4, g, e, case["n"],
                                     case["k"])
    else:
        width = (case["hq"] + 2 * case["hk"]) * case["d"]   # queries, keys, values
        st["x"] = torch.randn((case["tokens"], width), generator=g, device="cuda").to(_dtype(case["dtype"]))
        st["gq"] = (1 + 0.1 * torch.randn((case["d"],), generator=g, device="cuda")).to(_dtype(case["dtype"]))
        st["gk"] = (1 + 0.1 * torch.randn((case["d"],), generator=g, device="cuda")).to(_dtype(case["dtype"]))
        half = case["rot"] // 2
        freq = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        angle = torch.arange(case["tokens"] + 64, device="cuda", dtype=torch.float64)[:, None] * freq
        st["cos"], st["sin"] = angle.cos().float(), angle.sin().float()
        # a sequence that begins somewhere in the tables
        first = int(torch.randint(0, 64, (1,), generator=g, device="cuda"))
        st["pos"] = torch.arange(first, first + case["tokens"], device="cuda", dtype=torch.int32)
    return st


def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


# ---- plain forms ----------------------------------------------------------

def _plain_quantize(st):
    x = st["x"].float()
    s = x.abs().amax(dim=1, keepdim=True) / 127.0
    q = torch.round(x / s).clamp(-127, 127)
    q = torch.where(s > 0, q, torch.zeros_like(q))
    return {"values": (q * s).to(torch.bfloat16), "scales": s}


def _plain_gemm(st):
    y = st["a"].float() @ st["w"].float().t()
    y = y * st["sa"][:, None] * st["sw"]
    if st["bias"] is not None:
        y = y + st["bias"].float()
    return y.to(torch.bfloat16)


def _plain_mxfp4(codes, scales):
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=codes.device)
    v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], dim=2)
    v = v.view(codes.shape[0], -1, 32) * torch.exp2(scales.float() - 127.0)[:, :, None]
    return v.view(codes.shape[0], -1)


def _plain_grouped(st):
    c = st["case"]
    e, n, off = c["experts"], c["n"], st["offsets"]
    m = torch.arange(st["a"].shape[0], device=off.device, dtype=torch.int32)
    who = torch.searchsorted(off[1:], m, right=True)
    w, sw = st["w"].view(e, n, -1), st["sw"].view(e, n, -1)
    few = m.numel() < e
    if few:   # fewer rows than experts: take each row's own weights only
        w, sw = w[who], sw[who]
    w, sw = w.flatten(0, 1), sw.flatten(0, 1)
    if c["pair"] == "i8":
        a, w = st["a"].float() * st["sa"][:, None], w.float() * sw
    else:
        a = _plain_mxfp4(st["a"], st["sa"]) if c["pair"] == "mx4" else st["a"].float()
        w = _plain_mxfp4(w, sw)
    w = w.view(-1, n, a.shape[1]).transpose(1, 2)
    if few:
        return torch.bmm(a[:, None, :], w)[:, 0].to(torch.bfloat16)
    # every expert's rows padded to the largest group: one batched product
    slot = torch.arange(st["cap"], device=a.device)
    rows = (off[:-1, None] + slot).clamp_max(a.shape[0] - 1)
    return torch.bmm(a[rows], w)[who, m - off[who]].to(torch.bfloat16)


def _plain_qknorm(st):
    c = st["case"]
    t, d, r = c["tokens"], c["d"], c["rot"]
    cos, sin = st["cos"][st["pos"]][:, None, :], st["sin"][st["pos"]][:, None, :]

    def head(x, gain):
        x = x.float().view(t, -1, d)
        x = x * torch.rsqrt((x * x).mean(dim=2, keepdim=True) + 1e-6) * gain.float()
        if c["pairs"] == "half":
            a, b = x[:, :, :r // 2], x[:, :, r // 2:r]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=2)
        else:
            a, b = x[:, :, 0:r:2], x[:, :, 1:r:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=3).view(t, -1, r)
        return torch.cat([turned, x[:, :, r:]], dim=2).to(st["x"].dtype)

    nq, nk = c["hq"] * d, c["hk"] * d
    return {"q": head(st["x"][:, :nq], st["gq"]), "k": head(st["x"][:, nq:nq + nk], st["gk"])}


_plain = {"quantize": _plain_quantize, "gemm": _plain_gemm, "grouped": _plain_grouped,
          "qknorm": _plain_qknorm}


# ---- through the package --------------------------------------------------

def _own_quantize(st):
    import fp8_quantized_linear_mxq_amd as mxq
    q = mxq.quantize(st["x"], mxq.INT8)
    values = torch.empty(q.codes.shape, dtype=torch.bfloat16, device=q.codes.device)
    torch.mul(q.codes.view(torch.int8), q.scales, out=values)
    return {"values": values, "scales": q.scales}


def _own_gemm(st):
    import fp8_quantized_linear_mxq_amd as mxq
    return mxq.gemm(mxq.int8_operand(st["a"], st["sa"]), mxq.int8_operand(st["w"], st["sw"]),
                    bias=st["bias"])


def _own_grouped(st):
    import fp8_quantized_linear_mxq_amd as mxq
    c = st["case"]
    rows, wrows, k = st["a"].shape[0], st["w"].shape[0], c["k"]
    if c["pair"] == "i8":
        a, w = mxq.int8_operand(st["a"], st["sa"]), mxq.int8_operand(st["w"], st["sw"])
    else:
        w = mxq.QTensor(mxq.MXFP4, wrows, k, st["w"], st["sw"])
        a = (mxq.QTensor(mxq.MXFP4, rows, k, st["a"], st["sa"]) if c["pair"] == "mx4"
             else mxq.bf16_operand(st["a"]))
    return mxq.gemm_grouped(a, w, st["offsets"])


def _own_qknorm(st):
    import fp8_quantized_linear_mxq_amd as mxq
    c = st["case"]
    q, k = mxq.qk_norm_rope(st["x"], c["hq"], c["hk"], c["d"], st["gq"], st["gk"], st["cos"],
                            st["sin"], positions=st["pos"], eps=1e-6,
                            interleaved=c["pairs"] == "interleaved")
    return {"q": q, "k": k}


_own = {"quantize": _own_quantize, "gemm": _own_gemm, "grouped": _own_grouped,
        "qknorm": _own_qknorm}


# ---- what cannot be avoided, and the values in 64 bits --------------------

def work(case):
    op = case["op"]
    if op == "quantize":
        e = case["m"] * case["k"]
        return {"bytes": e * ((2 if case["dtype"] == "bf16" else 4) + 2) + 4 * case["m"],
                "flops": 4 * e}
    if op == "gemm":
        m, k, n = case["m"], case["k"], case["n"]
        return {"bytes": m * k + n * k + 4 * (m + n) + 2 * m * n + (2 * n if case["bias"] else 0),
                "flops": 2 * m * n * k}
    if op == "grouped":
        e, k, n = case["experts"], case["k"], case["n"]
        m = case["tokens"] * min(case["topk"], e)
        # experts that get rows, were all liked the same
        hit = e * (1 - (1 - min(case["topk"], e) / e) ** case["tokens"])
        per = {"i8": (k, k + 4), "mx4": (k / 2 + k / 32, k / 2 + k / 32), "w4a16": (2 * k, k / 2 + k / 32)}
        pa, pw = per[case["pair"]]
        return {"bytes": m * pa + hit * n * pw + 2 * m * n + 4 * (e + 1), "flops": 2 * m * n * k}
    t, heads, d = case["tokens"], case["hq"] + case["hk"], case["d"]
    size = 2 if case["dtype"] == "bf16" else 4
    return {"bytes": 2 * t * heads * d * size + t * (4 * case["rot"] + 4) + 2 * d * size,
            "flops": 7 * t * heads * d}


def _exact_mxfp4(codes, scales):
    lo, hi = (codes & 15).long(), (codes >> 4).long()
    c = torch.stack([lo, hi], dim=2).flatten(1)
    ex, man = (c >> 1) & 3, c & 1
    mag = torch.where(ex == 0, man.double() * 0.5, (1 + man.double() / 2) * torch.exp2(ex.double() - 1))
    v = torch.where(c >= 8, -mag, mag)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, dim=1)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = st["x"].double()
        s = (x.abs().max(dim=1, keepdim=True).values / 127).float().double()
        q = (x / torch.where(s == 0, torch.ones_like(s), s)).round().clamp(-127, 127)
        return {"values": q * s, "scales": s}
    if op == "gemm":
        y = (st["a"].double() * st["sa"].double()[:, None]) @ (st["w"].double() * st["sw"].double()[:, None]).T
        return y if st["bias"] is None else y + st["bias"].double()
    if op == "grouped":
        off = st["offsets"].tolist()
        out = torch.zeros((st["a"].shape[0], case["n"]), dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            if off[e] == off[e + 1]:
                continue
            rows, cols = slice(off[e], off[e + 1]), slice(e * case["n"], (e + 1) * case["n"])
            if case["pair"] == "i8":
                a = st["a"][rows].double() * st["sa"][rows].double()[:, None]
                w = st["w"][cols].double() * st["sw"][cols].double()[:, None]
            else:
                a = _exact_mxfp4(st["a"][rows], st["sa"][rows]) if case["pair"] == "mx4" else st["a"][rows].double()
                w = _exact_mxfp4(st["w"][cols], st["sw"][cols])
            out[rows] = a @ w.T
        return out
    t, d, r, nq = case["tokens"], case["d"], case["rot"], case["hq"] * case["d"]
    turn = torch.complex(st["cos"].double(), st["sin"].double())[st["pos"].long()][:, None]
    got = {}
    for name, x, gain in (("q", st["x"][:, :nq], st["gq"]),
                          ("k", st["x"][:, nq:nq + case["hk"] * d], st["gk"])):
        x = x.double().reshape(t, -1, d)
        x = x / (x.square().sum(dim=2, keepdim=True) / d + 1e-6).sqrt() * gain.double()
        if case["pairs"] == "half":
            z = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) * turn
            head = torch.cat([z.real, z.imag], dim=2)
        else:
            z = torch.complex(x[..., 0:r:2].contiguous(), x[..., 1:r:2].contiguous()) * turn
            head = torch.view_as_real(z).flatten(2)
        got[name] = torch.cat([head, x[..., r:]], dim=2)
    return got
