"""One whole decoder block: the library's projections, norms of queries and keys, and the MoE layer in one call.

    python examples/decoder_block.py [--tokens 64] [--steps 8]

Serving (`DecoderBlock.serve`), n tokens of one sequence, or the next one of it behind a cache:

    residual, x = block_norm(residual, the previous block's output)
    q, k, v     = linear(x) with a bias, one projection                 views into its rows
    q, k        = qk_norm_rope(q, k)                                    a norm a head, three axes of positions
    o           = linear(attention(q, k, v))                            the attention itself is plain torch
    residual, x = block_norm(residual, o)
    h           = linear(x), relu2;  d = residual + linear(h)           a dense branch beside the experts
    y           = d + routed experts + shared expert                    MoeLayer.layer_forward

Training (`DecoderBlock.train_step`): the attention's half towards a target for o, and the dense branch towards one
for y, with the experts, and what the second half does with the first half's result, left as they are.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from nvfp4_quantized_moe_topk_gb300 import api


class DecoderBlock:
    """H hidden channels, heads of D channels, I inner ones, E experts of which a token takes k, and one for all."""

    def __init__(self, H=256, heads=4, kv_heads=2, D=64, I=192, E=16, k=4, max_tokens=64, seed=0, device="cuda"):
        self.H, self.heads, self.kv_heads, self.D, self.I, self.E, self.k = H, heads, kv_heads, D, I, E, k
        g = torch.Generator(device="cpu").manual_seed(seed)
        dev = torch.device(device)

        def codes(*shape):  # two e2m1 codes a byte, e4m3 scales between 2^-4 and 2^2
            *lead, rows, cols = shape
            c = torch.randint(0, 256, (*lead, rows, cols // 2), generator=g, dtype=torch.uint8)
            s = (torch.randint(-4, 3, (*lead, rows, cols // 16), generator=g) + 7 << 3).to(torch.uint8)
            return c.to(dev), s.to(dev)

        def normal(*shape, scale=1.0, dtype=torch.bfloat16):
            return (torch.randn(shape, generator=g) * scale).to(dtype).to(dev)

        self.up, self.down = codes(E + 1, I, H), codes(E + 1, H, I)
        self.expert_global = torch.full((E + 1,), 2.0 ** -6, device=dev)
        self.layer = api.MoeLayer(H, I, E + 1, k + 1, max_tokens, *self.up, *self.down, self.expert_global,
                                  self.expert_global)
        self.router, self.router_bias = normal(E, H, scale=H ** -0.5), normal(E, scale=0.1, dtype=torch.float32)
        rows = (heads + 2 * kv_heads) * D
        self.qkv, self.qkv_bias = normal(rows, H, scale=H ** -0.5), normal(rows, scale=0.1)
        self.out = normal(H, heads * D, scale=(heads * D) ** -0.5)
        self.dense_up, self.dense_bias = normal(I, H, scale=H ** -0.5), normal(I, scale=0.1)
        self.dense_down = normal(H, I, scale=I ** -0.5)
        self.norm = {name: 1 + normal(H, scale=0.1, dtype=torch.float32)
                     for name in ("previous_post", "attention_pre", "attention_post", "moe_pre")}
        self.q_norm, self.k_norm = (1 + normal(D, scale=0.1) for _ in range(2))
        pairs = D // 2
        self.freq = (10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).float().to(dev)
        self.rope = dict(sections=[pairs - 2 * (pairs // 3), pairs // 3, pairs // 3], sections_interleaved=True)
        n, D3 = max_tokens, (self.heads + 2 * self.kv_heads) * D
        self.ws = {s: api.linear_workspace(n, *s) for s in {(H, D3), (heads * D, H), (H, I), (I, H)}}
        self.qk_ws = api.qk_workspace(n, heads, kv_heads, D)

    def split(self, rows):
        """A projection's rows as its queries, keys and values."""
        q, k = self.heads * self.D, self.kv_heads * self.D
        view = lambda t: t.unflatten(1, (-1, self.D))  # noqa: E731
        return view(rows[:, :q]), view(rows[:, q: q + k]), view(rows[:, q + k:])

    def attention(self, q, k, v):
        """Causal attention of the last len(q) of len(k) tokens, in fp32."""
        per = self.heads // self.kv_heads
        k, v = (t.float().repeat_interleave(per, 1) for t in (k, v))
        s = torch.einsum("qhd,khd->hqk", q.float(), k) * self.D ** -0.5
        s += torch.full(s.shape[1:], float("-inf"), device=s.device).triu(1 + k.shape[0] - q.shape[0])
        return torch.einsum("hqk,khd->qhd", s.softmax(-1), v).flatten(1)

    def serve(self, residual, previous, positions, cache=None):
        """residual, previous [n, H] bf16, positions [3, n] int32, cache (k, v) of the tokens before -> what each step
        left, by name."""
        n, dev = residual.shape[0], residual.device
        new = lambda c: torch.empty((n, c), dtype=torch.bfloat16, device=dev)  # noqa: E731
        r1, x1 = api.block_norm(residual, previous, None, self.norm["previous_post"], self.norm["attention_pre"],
                                new(self.H), new(self.H))
        qkv = api.linear(x1, self.qkv, new(self.qkv.shape[0]), self.qkv_bias)
        q, k, v = self.split(qkv)
        qr, kr = api.qk_norm_rope(q, k, torch.empty_like(q, memory_format=torch.contiguous_format),
                                  torch.empty_like(k, memory_format=torch.contiguous_format), positions, self.freq,
                                  self.q_norm, self.k_norm, **self.rope)
        ks, vs = (kr, v) if cache is None else (torch.cat([c, t]) for c, t in zip(cache, (kr, v)))
        a = self.attention(qr, ks, vs).bfloat16()
        o = api.linear(a, self.out, new(self.H))
        r2, x2 = api.block_norm(r1, o, None, self.norm["attention_post"], self.norm["moe_pre"], new(self.H),
                                new(self.H))
        z = new(self.I)
        h = api.linear(x2, self.dense_up, new(self.I), self.dense_bias, None, z, activation="relu2")
        d = api.linear(h, self.dense_down, new(self.H), None, r2)
        ids = torch.empty((n, self.k), dtype=torch.int32, device=dev)
        w = torch.empty((n, self.k), device=dev)
        y = self.layer.layer_forward(x2, self.router, new(self.H), d, self.router_bias, shared_experts=1, topk_ids=ids,
                                     topk_weights=w)
        return dict(r1=r1, x1=x1, qkv=qkv, qr=qr, kr=kr, ks=ks, vs=vs, a=a, o=o, r2=r2, x2=x2, z=z, h=h, d=d, ids=ids,
                    w=w, y=y)

    def train_step(self, residual, previous, positions, o_target, y_target, lr=0.0):
        """One step on (|o - o_target|^2 + |y - y_target|^2) / 2n.  Returns the two losses, the forward's tensors and
        the gradients by name."""
        s = self.serve(residual, previous, positions)
        n, dev = residual.shape[0], residual.device
        like = lambda t: torch.empty(t.shape, device=dev)  # noqa: E731
        half = lambda t: torch.empty(t.shape, dtype=torch.bfloat16, device=dev)  # noqa: E731
        g = dict(y=(s["y"].float() - y_target) / n, o=(s["o"].float() - o_target) / n)

        def back(name, d, x, weight, d_x=None, d_bias=None, z=None, activation="none"):
            _, g[name], _ = api.linear_backward(d, x, weight, z, d_x, like(weight), d_bias, activation=activation,
                                                workspace=self.ws[tuple(reversed(weight.shape))])

        g["h"], g["dense_bias"] = half(s["h"]), like(self.dense_bias)
        back("dense_down", g["y"], s["h"], self.dense_down, g["h"])
        back("dense_up", g["h"], s["x2"], self.dense_up, None, g["dense_bias"], s["z"], "relu2")

        g["a"], g["qkv_rows"], g["x1"], g["qkv_bias"] = half(s["a"]), half(s["qkv"]), half(s["x1"]), like(self.qkv_bias)
        back("out", g["o"], s["a"], self.out, g["a"])
        q, k, v = self.split(s["qkv"])
        leaves = [t.detach().requires_grad_(True) for t in (s["qr"], s["kr"], v)]
        g["qr"], g["kr"], dv = (t.contiguous() for t in torch.autograd.grad(self.attention(*leaves), leaves,
                                                                            g["a"].float()))
        d_q, d_k, d_v = self.split(g["qkv_rows"])
        d_v.copy_(dv)
        g["q_norm"], g["k_norm"] = like(self.q_norm), like(self.k_norm)
        api.qk_norm_rope_backward(g["qr"], g["kr"], q, k, d_q, d_k, positions, self.freq, self.q_norm, self.k_norm,
                                  g["q_norm"], g["k_norm"], workspace=self.qk_ws, **self.rope)
        back("qkv", g["qkv_rows"], s["x1"], self.qkv, g["x1"], g["qkv_bias"])
        for name in ("dense_down", "dense_up", "dense_bias", "out", "qkv", "qkv_bias", "q_norm", "k_norm"):
            getattr(self, name).sub_(lr * g[name])
        return float(0.5 * n * g["o"].square().sum()), float(0.5 * n * g["y"].square().sum()), s, g

    def close(self):
        self.layer.close()


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=64)
    p.add_argument("--steps", type=int, default=8)
    args = p.parse_args()
    n, dev = args.tokens, torch.device("cuda")
    block = DecoderBlock(max_tokens=n)
    rows = lambda n: torch.randn((n, block.H), device=dev).bfloat16()  # noqa: E731
    at = torch.arange(n, device=dev, dtype=torch.int32)
    positions = torch.stack([at, at // 8, at % 8])
    residual, previous = rows(n), rows(n)
    s = block.serve(residual, previous, positions)
    print(f"served {n} tokens: |y| {s['y'].float().norm():.2f}")
    one = block.serve(rows(1), rows(1), positions[:, -1:] + 1, (s["ks"], s["vs"]))
    print(f"and one more behind them: |y| {one['y'].float().norm():.2f}")
    o, y = s["o"].float() + 0.1 * rows(n).float(), s["y"].float() + 0.1 * rows(n).float()
    for i in range(args.steps):
        lo, ly, *_ = block.train_step(residual, previous, positions, o, y, lr=0.002)
        print(f"step {i}: attention's half {lo:.5f}, dense branch {ly:.5f}")
    assert api.linear_device_error() == 0 and block.layer.device_error() == 0
    block.close()


if __name__ == "__main__":
    main()
