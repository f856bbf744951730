"""One transformer block's MoE half through the library's operators.

    python examples/moe_block.py [--tokens 64] [--steps 8]

Serving (`MoeBlock.serve`), one batch of tokens of several requests:

    residual, x = block_norm(residual, attention's output)     the norms around the previous block, one call
    ids, w      = router_topk(x router^T)
    y           = x shared + the request's adapter on it         nvfp4_matmul, lora_apply
    y          += the experts' weighted outputs                  MoeLayer.forward
    residual, x = block_norm(residual, y)                        before the next block

Training the router over frozen experts (`MoeBlock.train_step`): the balance
loss next to a squared error at the block's output, and the gradient back
through the norm, the top-k weights and the loss to the router's weights.

Every tensor that a step needs is made once, workspaces too.  The weights here
are random; the library's calls run on the current stream.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from nvfp4_quantized_moe_topk_gb300 import api


class MoeBlock:
    """H hidden channels, I inner ones, E experts of which a token takes k, L adapters of ranks up to R."""

    def __init__(self, H=512, I=256, E=16, k=4, L=4, R=16, max_tokens=64, seed=0, device="cuda"):
        self.H, self.E, self.k, self.L = H, E, k, L
        g = torch.Generator(device="cpu").manual_seed(seed)
        dev = torch.device(device)

        def codes(*shape):  # two e2m1 codes a byte, e4m3 scales between 2^-4 and 2^2
            *lead, rows, cols = shape
            c = torch.randint(0, 256, (*lead, rows, cols // 2), generator=g, dtype=torch.uint8)
            s = (torch.randint(-4, 3, (*lead, rows, cols // 16), generator=g) + 7 << 3).to(torch.uint8)
            return c.to(dev), s.to(dev)

        def normal(*shape, scale=1.0, dtype=torch.float32):
            return (torch.randn(shape, generator=g) * scale).to(dtype).to(dev)

        self.up, self.down, self.shared = codes(E, I, H), codes(E, H, I), codes(H, H)
        self.expert_global = torch.full((E,), 2.0 ** -6, device=dev)
        self.shared_global = 2.0 ** -6
        self.layer = api.MoeLayer(H, I, E, k, max_tokens, *self.up, *self.down, self.expert_global, self.expert_global)
        self.router, self.bias = normal(E, H, scale=H ** -0.5), normal(E, scale=0.1)
        self.a = normal(L, R, H, scale=H ** -0.5, dtype=torch.bfloat16)
        self.b = normal(L, H, R, scale=R ** -0.5, dtype=torch.bfloat16)
        self.ranks = torch.tensor([R - (l % 2) * (R // 2) for l in range(L)], dtype=torch.int32, device=dev)
        self.scale = torch.full((L,), 2.0, device=dev)
        self.gate = normal(H, scale=0.5)
        self.norm = {name: 1 + normal(H, scale=0.1) for name in ("attention_post", "moe_pre", "moe_post", "next_pre")}
        self.branch_scale = 0.5
        self.lora_ws = api.lora_workspace(max_tokens, L)
        self.router_ws = api.router_workspace(max_tokens, E, max_tokens)
        self.norm_ws = api.block_norm_workspace(max_tokens, H)

    def route(self, x, n):
        logits = x.float() @ self.router.T
        ids = torch.empty((n, self.k), dtype=torch.int32, device=x.device)
        w = torch.empty((n, self.k), dtype=torch.float32, device=x.device)
        api.router_topk(logits, self.bias, ids, w)
        return logits, ids, w

    def shared_projection(self, x, adapter_ids):
        """The shared NVFP4 projection with each token's adapter on it, bf16."""
        y = torch.empty((x.shape[0], self.H), device=x.device)
        api.nvfp4_matmul(x, *self.shared, self.shared_global, y, 0)
        out = torch.empty_like(x)
        return api.lora_apply(x, adapter_ids, self.a, self.b, y, out, scale=self.scale, ranks=self.ranks,
                              workspace=self.lora_ws)

    def serve(self, residual, attention, adapter_ids):
        """residual, attention [n, H] bf16, adapter_ids [n] int32 (-1: none) -> what each step left, by name."""
        n = residual.shape[0]
        r1, x1 = api.block_norm(residual, attention, self.gate, self.norm["attention_post"], self.norm["moe_pre"],
                                torch.empty_like(residual), torch.empty_like(residual), gate_sigmoid=True)
        _, ids, w = self.route(x1, n)
        shared = self.shared_projection(x1, adapter_ids)
        y = shared.clone()
        self.layer.forward(x1, ids, w, y)
        r2, x2 = api.block_norm(r1, y, None, self.norm["moe_post"], self.norm["next_pre"], torch.empty_like(residual),
                                torch.empty_like(residual), branch_scale=self.branch_scale)
        return dict(r1=r1, x1=x1, ids=ids, w=w, shared=shared, y=y, r2=r2, x2=x2)

    def expert_outputs(self, x, ids):
        """[k, n, H]: each token's experts one by one (frozen: no gradient goes into them)."""
        n = x.shape[0]
        out = torch.zeros((self.k, n, self.H), dtype=torch.bfloat16, device=x.device)
        for j in range(self.k):
            one = torch.zeros((n, self.k), device=x.device)
            one[:, j] = 1
            self.layer.forward(x, ids, one, out[j])
        return out

    def train_step(self, residual, x, adapter_ids, target, seq_offsets, mask, coef=0.01, lr=0.0):
        """One step of the router on 0.5 |residual_out - target|^2 / n + balance loss, residual [n, H] fp32 and x
        [n, H] bf16.  Returns the two losses and the gradients of the router's weights and bias."""
        n, dev = x.shape[0], x.device
        logits, ids, w = self.route(x, n)
        seqs = seq_offsets.numel() - 1
        balance = torch.empty(1, device=dev)
        counts = torch.empty((seqs, self.E), dtype=torch.int32, device=dev)
        sums = torch.empty((seqs, self.E), device=dev)
        tokens = torch.empty(seqs + 1, dtype=torch.int32, device=dev)
        router = dict(coef=coef, mask=mask, seq_offsets=seq_offsets, workspace=self.router_ws)
        api.balance_loss(logits, self.bias, ids, balance, counts, sums, tokens, **router)

        y = self.shared_projection(x, adapter_ids)
        self.layer.forward(x, ids, w, y)
        norm = dict(branch_scale=self.branch_scale)
        rstd = torch.empty(n, device=dev)
        out, _ = api.block_norm(residual, y, None, self.norm["moe_post"], None, torch.empty_like(residual), None, rstd,
                                **norm)
        error = out - target
        d_y = torch.empty_like(y)
        api.block_norm_backward(error / n, None, out, y, None, self.norm["moe_post"], None, rstd, None, None, d_y,
                                workspace=self.norm_ws, **norm)
        d_w = torch.einsum("nh,knh->nk", d_y.float(), self.expert_outputs(x, ids).float()).contiguous()
        d_logits, d_bias = torch.empty_like(logits), torch.empty_like(self.bias)
        api.router_backward(logits, self.bias, ids, w, d_w, counts, tokens, d_logits, d_bias, **router)
        d_router = d_logits.T @ x.float()
        self.router -= lr * d_router
        self.bias -= lr * d_bias
        return float(0.5 * (error * error).sum() / n), float(balance), d_router, d_bias

    def close(self):
        self.layer.close()


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=64)
    p.add_argument("--steps", type=int, default=8)
    args = p.parse_args()
    n, dev = args.tokens, torch.device("cuda")
    block = MoeBlock(max_tokens=n)
    residual, attention = (torch.randn((n, block.H), device=dev).bfloat16() for _ in range(2))
    requests = (torch.arange(n, device=dev, dtype=torch.int32) // 8) % (block.L + 1) - 1
    step = block.serve(residual, attention, requests)
    print(f"served {n} tokens: |residual| {step['r2'].float().norm():.2f}, |x| {step['x2'].float().norm():.2f}")
    offsets = torch.tensor([0, n // 3, n], dtype=torch.int32, device=dev)
    mask = torch.ones(n, dtype=torch.bool, device=dev)
    target = step["r1"].float() + 0.5 * torch.randn((n, block.H), device=dev)
    for i in range(args.steps):
        error, balance, *_ = block.train_step(step["r1"].float(), step["x1"], requests, target, offsets, mask, lr=0.05)
        print(f"step {i}: error {error:.5f}, balance loss {balance:.5f}")
    assert api.lora_device_error() == 0 and block.layer.device_error() == 0
    block.close()


if __name__ == "__main__":
    main()
