"""The operators around the layer together, as examples/moe_block.py runs them: each step of serving against 64 bits
from the tensors that the step before it left, and a training step's gradient against automatic differentiation of the
formulas in 64 bits.

Tolerances.  A bf16 result is one rounding of an fp32 one: 2^-8 of its value covers half a unit in the last place with
room for the fp32 sums, which get 2^-15 of the same formula with every term's absolute value (an adapter's inner result
keeps 16 bits).  The layer has its own bound (helpers.layer_tolerance_check).  The gradient passes through three bf16
tensors (the experts' outputs, the block's output and its gradient), each 2^-9 of its value, and the norm's backward pass
doubles what enters it: 2^-6 of the gradient's formula with absolute values."""
import os
import sys

import numpy as np
import pytest

import helpers
import oracle
from nvfp4_quantized_moe_topk_gb300 import workload as W

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

ROUND, SUMS, GRAD = 2.0 ** -8, 2.0 ** -15, 2.0 ** -6


@pytest.fixture(scope="module")
def dev():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return torch.device("cuda:0")


def _close(got, want, scale):
    err = (got.double().cpu() - want).abs()
    assert bool((err <= ROUND * want.abs() + SUMS * scale).all()), float((err / scale.clamp(min=1e-30)).max())


def _norm(u, weight):
    return u * (u.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * weight


def _bits(t):
    import torch

    return t.cpu().view(torch.int16).numpy().view(np.uint16)


@pytest.mark.parametrize("n", [1, 7, 200, 1500])
def test_serving_step_by_step(dev, n):
    import torch

    import moe_block

    block = moe_block.MoeBlock(max_tokens=n, seed=n)
    g = torch.Generator().manual_seed(n)
    residual, attention = (torch.randn((n, block.H), generator=g).bfloat16().to(dev) for _ in range(2))
    ids = (torch.arange(n, device=dev, dtype=torch.int32) // 5) % (block.L + 1) - 1
    out = block.serve(residual, attention, ids)
    torch.cuda.synchronize()
    d = {k: v.double().cpu() for k, v in out.items() if k != "ids"}
    p = {k: v.double().cpu() for k, v in block.norm.items()}

    z = torch.sigmoid(block.gate.double().cpu()) * _norm(attention.double().cpu(), p["attention_post"])
    u = residual.double().cpu() + z
    scale = residual.double().cpu().abs() + z.abs()
    _close(out["r1"], u, scale)
    ru = (u.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
    _close(out["x1"], u * ru * p["moe_pre"], scale * ru * p["moe_pre"].abs())

    logits = d["x1"] @ block.router.double().cpu().T + block.bias.double().cpu()
    picked = torch.gather(logits, 1, out["ids"].long().cpu())
    assert bool((d["w"] - torch.softmax(picked, -1)).abs().max() <= 1e-4)

    weight = torch.from_numpy(oracle.dequant(block.shared[0].cpu().numpy(), block.shared[1].cpu().numpy(), block.H,
                                             block.H)) * block.shared_global
    want, scale = d["x1"] @ weight.T, d["x1"].abs() @ weight.abs().T
    for l in range(block.L):
        r, rows = int(block.ranks[l]), (ids == l).cpu()
        a, b = block.a[l, :r].double().cpu(), block.b[l, :, :r].double().cpu()
        want[rows] += float(block.scale[l]) * (d["x1"][rows] @ a.T) @ b.T
        scale[rows] += float(block.scale[l]) * (d["x1"][rows].abs() @ a.abs().T) @ b.abs().T
    _close(out["shared"], want, scale)

    if n <= 200:
        glob = block.expert_global.cpu().numpy()
        wl = W.Workload("block", n, block.H, 256, block.E, block.k, _bits(out["x1"]), out["ids"].cpu().numpy(),
                        out["w"].cpu().numpy(), *(t.cpu().numpy() for t in (*block.up, *block.down)), glob, glob,
                        _bits(out["shared"]))
        ok, err, rms = helpers.layer_tolerance_check(_bits(out["y"]), oracle.moe_forward(wl, out_f64=True).out_f64)
        assert ok, (err, rms)

    z = block.branch_scale * _norm(d["y"], p["moe_post"])
    u, scale = d["r1"] + z, d["r1"].abs() + z.abs()
    _close(out["r2"], u, scale)
    ru = (u.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
    _close(out["x2"], u * ru * p["next_pre"], scale * ru * p["next_pre"].abs())
    block.close()


@pytest.mark.parametrize("n", [12, 300])
def test_router_gradient_of_a_training_step(dev, n):
    import torch

    import moe_block

    coef = 0.05
    block = moe_block.MoeBlock(max_tokens=n, seed=n)
    g = torch.Generator().manual_seed(n)
    x = torch.randn((n, block.H), generator=g).bfloat16().to(dev)
    residual, target = (torch.randn((n, block.H), generator=g).to(dev) for _ in range(2))
    requests = (torch.arange(n, device=dev, dtype=torch.int32) // 5) % (block.L + 1) - 1
    ends = [0, n // 3, n]
    mask = torch.rand(n, generator=g) > 0.1
    error, balance, d_router, d_bias = block.train_step(
        residual, x, requests, target, torch.tensor(ends, dtype=torch.int32, device=dev), mask.to(dev), coef=coef)
    _, ids, _ = block.route(x, n)
    outs = block.expert_outputs(x, ids).double().cpu()
    shared = block.shared_projection(x, requests).double().cpu()
    ids, x, residual, target = ids.long().cpu(), x.double().cpu(), residual.double().cpu(), target.double().cpu()

    router, bias = (t.double().cpu().requires_grad_() for t in (block.router, block.bias))
    logits = x @ router.T + bias
    logits.retain_grad()
    w = torch.softmax(torch.gather(logits, 1, ids), -1)
    y = shared + (w.T[:, :, None] * outs).sum(0)
    y.retain_grad()
    out = residual + block.branch_scale * _norm(y, block.norm["moe_post"].double().cpu())
    want_error = 0.5 * (out - target).square().sum() / n
    prob = torch.softmax(logits, -1)
    load = torch.zeros((n, block.E), dtype=torch.float64)  # the balance loss's gradient at each probability
    for lo, hi in zip(ends, ends[1:]):
        on = torch.zeros(n, dtype=torch.bool)
        on[lo:hi] = mask[lo:hi]
        counts = torch.bincount(ids[on].flatten(), minlength=block.E).double()
        load[on] = coef * block.E / (int(mask.sum()) * block.k) * counts / int(on.sum())
    want_balance = (load * prob).sum()
    (want_error + want_balance).backward()
    want_error, want_balance = want_error.item(), want_balance.item()
    assert abs(error - want_error) <= GRAD * want_error
    assert abs(balance - want_balance) <= 1e-4 * want_balance

    dw = (y.grad.abs()[None] * outs.abs()).sum(-1).T
    dz = w * (dw + (w * dw).sum(-1, keepdim=True))
    scale = prob * (load + (load * prob).sum(-1, keepdim=True))
    scale = scale.detach().scatter_add(1, ids, dz.detach())
    assert bool(((d_bias.double().cpu() - bias.grad).abs() <= GRAD * scale.sum(0)).all())
    assert bool(((d_router.double().cpu() - router.grad).abs() <= GRAD * (scale.T @ x.abs())).all())
    block.close()
