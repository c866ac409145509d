"""One transformer block of routed experts on quantized weights, for serving.

  x -> int8 rows -> QKV product -> head norms + rotation -> attention
    -> int8 rows -> output product -> + x = h
  h -> router -> rows sorted by expert -> quantized rows -> grouped up product
    -> gate -> quantized rows -> grouped down product -> weighted sum + h

The norms in front of the two halves are left out.  Experts run on one of three
pairs of operands: int8 x int8, MXFP4 x MXFP4, or bf16 x MXFP4.  Attention
itself, the router and the gate are plain torch.

  python examples/expert_block.py [--tokens 256] [--experts 16] [--pair int8|mxfp4|w4a16]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_quantized_linear_mxq_amd as mxq

FORMATS = {"int8": (mxq.INT8, mxq.INT8), "mxfp4": (mxq.MXFP4, mxq.MXFP4), "w4a16": (mxq.BF16, mxq.MXFP4)}


class ExpertBlock:
    def __init__(self, width=1024, heads=8, kv_heads=2, head_dim=128, experts=16, topk=4, hidden=512,
                 pair="int8", n_pos=4096, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        draw = lambda *s: torch.randn(s, generator=g, device="cuda")
        self.heads, self.kv_heads, self.d, self.n_experts, self.topk = heads, kv_heads, head_dim, experts, topk
        self.hidden = hidden
        self.act, wfmt = FORMATS[pair]
        # weights are quantized once; bf16 sources only to keep the draw small
        weight = lambda n, k, fmt: mxq.quantize((draw(n, k) / k ** 0.5).bfloat16(), fmt)
        self.wqkv = weight((heads + 2 * kv_heads) * head_dim, width, mxq.INT8)
        self.wout = weight(width, heads * head_dim, mxq.INT8)
        self.w_up = weight(experts * 2 * hidden, width, wfmt)      # [expert][gate rows, up rows]
        self.w_down = weight(experts * width, hidden, wfmt)
        self.router = draw(experts, width) / width ** 0.5
        self.q_gain = (1 + 0.1 * draw(head_dim)).bfloat16()
        self.k_gain = (1 + 0.1 * draw(head_dim)).bfloat16()
        angle = torch.arange(n_pos, device="cuda")[:, None] * \
            1e4 ** (-torch.arange(0, head_dim, 2, device="cuda") / head_dim)
        self.cos, self.sin = angle.cos(), angle.sin()

    def operand(self, x):
        return mxq.bf16_operand(x) if self.act == mxq.BF16 else mxq.quantize(x, self.act)

    def attention(self, x, positions):
        """h [tokens, width] of one sequence: causal attention and the residual."""
        t = x.shape[0]
        qkv = mxq.gemm(mxq.quantize(x, mxq.INT8), self.wqkv)
        q, k = mxq.qk_norm_rope(qkv, self.heads, self.kv_heads, self.d, self.q_gain, self.k_gain,
                                self.cos, self.sin, positions=positions)
        v = qkv[:, -self.kv_heads * self.d:].view(t, self.kv_heads, self.d)
        o = causal(q.float(), k.float(), v.float()).bfloat16()
        return x + mxq.gemm(mxq.quantize(o, mxq.INT8), self.wout)

    def route(self, h):
        p, pick = (h.float() @ self.router.t()).softmax(1).topk(self.topk, dim=1)
        return p / p.sum(1, keepdim=True), pick

    def experts(self, h, p, pick):
        t = h.shape[0]
        flat = pick.flatten()
        order = flat.argsort(stable=True)                       # rows of an expert lie together
        bounds = torch.arange(self.n_experts + 1, device="cuda")
        offsets = torch.searchsorted(flat[order], bounds, out_int32=True)   # stays on the device
        up = mxq.gemm_grouped(self.operand(h[order // self.topk]), self.w_up, offsets)
        act = torch.nn.functional.silu(up[:, :self.hidden].float()) * up[:, self.hidden:].float()
        down = mxq.gemm_grouped(self.operand(act.bfloat16()), self.w_down, offsets)
        back = torch.empty_like(order)
        back[order] = torch.arange(order.numel(), device="cuda")
        y = (down[back].view(t, self.topk, -1).float() * p[:, :, None]).sum(1)
        return (h.float() + y).bfloat16()

    def __call__(self, x, positions):
        h = self.attention(x, positions)
        return self.experts(h, *self.route(h))


def causal(q, k, v):
    """softmax(q k^T / sqrt(d)) v with shared key heads; [tokens, heads, d] -> [tokens, heads * d]."""
    t, heads, d = q.shape
    mask = torch.full((t, t), float("-inf"), device=q.device, dtype=q.dtype).triu(1)
    out = []
    for i in range(heads):
        j = i * k.shape[1] // heads
        out.append(((q[:, i] @ k[:, j].t()) * d ** -0.5 + mask).softmax(1) @ v[:, j])
    return torch.cat(out, 1)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=256)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--pair", choices=FORMATS, default="int8")
    args = ap.parse_args()
    block = ExpertBlock(experts=args.experts, pair=args.pair)
    x = torch.randn(args.tokens, 1024, device="cuda").bfloat16()
    pos = torch.arange(args.tokens, dtype=torch.int32, device="cuda")
    y = block(x, pos)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(20):
        y = block(x, pos)
    torch.cuda.synchronize()
    print(f"{args.pair}: {args.tokens} tokens, {args.experts} experts: "
          f"{(time.perf_counter() - t0) / 20 * 1e3:.3f} ms a block, output rms {y.float().square().mean().sqrt():.3f}")


if __name__ == "__main__":
    main()
