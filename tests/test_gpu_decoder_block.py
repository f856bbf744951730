"""Projections, norms of queries and keys with rotation, and the whole layer together, as examples/decoder_block.py runs
them: each step of serving, and each step of a training step's backward pass, against 64 bits from the tensors that the
step before it left.

Tolerances.  A bf16 result is one rounding of an fp32 one: 2^-8 of its value covers half a unit in the last place with
room for the fp32 sums, which get 2^-15 of the same formula with every term's absolute value: a product of C <= 256
terms is within (C / 16 + 16) 2^-22 = 2^-17 of it, a norm or a turn within 2^-17 (256 values; 64 units of 2^-24), a
product over n <= 300 rows within 2^-16.  relu2 doubles what its argument is off by.  A bf16 gradient of a product is
summed from the incoming gradient rounded to bf16: 2^-8 of the formula with absolute values.  The layer has its own bound
(helpers.layer_tolerance_check)."""
import os
import sys

import numpy as np
import pytest

import helpers
import oracle
from nvfp4_quantized_moe_topk_gb300 import workload as W

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

import decoder_block  # noqa: E402

ROUND, SUMS, D = 2.0 ** -8, 2.0 ** -15, torch.float64


def _close(got, want, scale, rounding=ROUND, terms=0.0):
    """terms: what each term may be off by beyond the sums."""
    err = (got.to(D) - want).abs()
    bound = rounding * want.abs() + (SUMS + terms) * scale
    assert bool((err <= bound).all()), float((err / bound.clamp(min=1e-30)).max())


def _product(got, x, w, bias=0.0, **kw):
    x, w = x.to(D), w.to(D)
    _close(got, x @ w.t() + bias, x.abs() @ w.abs().t() + abs(bias), **kw)


def _norms(r_out, x_out, residual, branch, post, pre):
    r, b, post, pre = (t.to(D) for t in (residual, branch, post, pre))
    z = b * (b.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * post
    u, size = r + z, r.abs() + z.abs()
    _close(r_out, u, size)
    ru = (u.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
    _close(x_out, u * ru * pre, size * ru * pre.abs())


def _turns(block, positions):
    """cos and sin [n, 1, pairs] of each pair's axis, which take turns."""
    s, pairs = block.rope["sections"], block.D // 2
    axis = [i % 3 if i // 3 < s[i % 3] else 0 for i in range(pairs)]
    angle = positions[axis].to(D).t() * block.freq.to(D)
    return torch.cos(angle)[:, None], torch.sin(angle)[:, None]


def _qk(block, h, weight, positions):
    """A head's norm and turn, and the sizes of its terms."""
    c, s = _turns(block, positions)
    y = h * (h.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * weight
    a, b = y.chunk(2, -1)
    size = a.abs() + b.abs()
    return torch.cat([a * c - b * s, b * c + a * s], -1), torch.cat([size, size], -1)


def _inputs(block, n, seed):
    g = torch.Generator().manual_seed(seed)
    rows = [torch.randn((n, block.H), generator=g).cuda() for _ in range(4)]
    positions = torch.randint(0, 5000, (3, n), generator=g, dtype=torch.int32).cuda()
    return rows[0].bfloat16(), rows[1].bfloat16(), positions, rows[2], rows[3]


def _bits(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


def _check_served(block, s, residual, previous, positions):
    p, n = block.norm, residual.shape[0]
    _norms(s["r1"], s["x1"], residual, previous, p["previous_post"], p["attention_pre"])
    _product(s["qkv"], s["x1"], block.qkv, block.qkv_bias.to(D))
    q, k, _ = block.split(s["qkv"])
    _close(s["qr"], *_qk(block, q.to(D), block.q_norm.to(D), positions))
    _close(s["kr"], *_qk(block, k.to(D), block.k_norm.to(D), positions))
    _product(s["o"], s["a"], block.out)
    _norms(s["r2"], s["x2"], s["r1"], s["o"], p["attention_post"], p["moe_pre"])
    x, w = s["x2"].to(D), block.dense_up.to(D)
    z, size = x @ w.t() + block.dense_bias.to(D), x.abs() @ w.abs().t() + block.dense_bias.to(D).abs()
    _close(s["z"], z, size)
    _close(s["h"], z.clamp(min=0).square(), 2 * (z.abs() + SUMS * size) * size)
    _product(s["d"], s["h"], block.dense_down, s["r2"].to(D))
    logits = x @ block.router.to(D).t() + block.router_bias.to(D)
    picked = torch.gather(logits, 1, s["ids"].long())
    assert bool(((s["w"] - torch.softmax(picked, -1)).abs() <= 1e-4).all())
    least = picked.min(1).values
    others = logits.scatter(1, s["ids"].long(), -torch.inf).max(1).values
    assert bool((others <= least + 1e-4).all())
    ids = torch.cat([s["ids"], s["ids"].new_full((n, 1), block.E)], 1)
    weights = torch.cat([s["w"], s["w"].new_ones((n, 1))], 1)
    glob = block.expert_global.cpu().numpy()
    wl = W.Workload("block", n, block.H, block.I, block.E + 1, block.k + 1, _bits(s["x2"]), ids.cpu().numpy(),
                    weights.cpu().numpy(), *(t.cpu().numpy() for t in (*block.up, *block.down)), glob, glob,
                    _bits(s["d"]))
    ok, err, rms = helpers.layer_tolerance_check(_bits(s["y"]), oracle.moe_forward(wl, out_f64=True).out_f64)
    assert ok, (err, rms)


@pytest.mark.parametrize("n", [1, 7, 61, 300])
def test_serving_step_by_step(n):
    block = decoder_block.DecoderBlock(max_tokens=max(n, 8), seed=n)
    residual, previous, positions, *_ = _inputs(block, n, n)
    s = block.serve(residual, previous, positions)
    _check_served(block, s, residual, previous, positions)
    residual, previous, positions, *_ = _inputs(block, 1, n + 1)  # the next token behind them
    _check_served(block, block.serve(residual, previous, positions, (s["ks"], s["vs"])), residual, previous, positions)
    block.close()


@pytest.mark.parametrize("n", [1, 61, 300])
def test_backward_step_by_step(n):
    block = decoder_block.DecoderBlock(max_tokens=n, seed=n)
    residual, previous, positions, o_target, y_target = _inputs(block, n, n)
    _, _, s, g = block.train_step(residual, previous, positions, o_target, y_target)
    fp32 = dict(rounding=2.0 ** -24)
    t = lambda m: m.to(D).t()  # noqa: E731
    _product(g["dense_down"], t(g["y"]), t(s["h"]), **fp32)
    _product(g["h"], g["y"], t(block.dense_down), terms=ROUND)
    dz = g["h"].to(D) * 2 * s["z"].to(D).clamp(min=0)
    _product(g["dense_up"], dz.t(), t(s["x2"]), **fp32)
    _close(g["dense_bias"], dz.sum(0), dz.abs().sum(0), **fp32)
    _product(g["out"], t(g["o"]), t(s["a"]), **fp32)
    _product(g["a"], g["o"], t(block.out), terms=ROUND)
    q, k, _ = block.split(s["qkv"])
    d_q, d_k, _ = block.split(g["qkv_rows"])
    for h, w, turned, d, dw in ((q, block.q_norm, g["qr"], d_q, g["q_norm"]), (k, block.k_norm, g["kr"], d_k, g["k_norm"])):
        h, w = h.to(D).requires_grad_(True), w.to(D).requires_grad_(True)
        y, _ = _qk(block, h, w, positions)
        want_h, want_w = torch.autograd.grad(y, (h, w), turned.to(D))
        h, w = h.detach(), w.detach().abs()
        r = (h.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
        a, b = turned.to(D).abs().chunk(2, -1)
        size = torch.cat([a + b, a + b], -1)
        _close(d, want_h, r * (w * size + (h * r).abs() * (w * size * (h * r).abs()).mean(-1, keepdim=True)))
        _close(dw, want_w, (size * (h * r).abs()).sum((0, 1)), **fp32)
    _product(g["qkv"], t(g["qkv_rows"]), t(s["x1"]), **fp32)
    _close(g["qkv_bias"], g["qkv_rows"].to(D).sum(0), g["qkv_rows"].to(D).abs().sum(0), **fp32)
    _product(g["x1"], g["qkv_rows"], t(block.qkv), terms=ROUND)
    block.close()


@pytest.mark.parametrize("name", ["qkv", "q_norm", "dense_up", "dense_bias", "out", "dense_down"])
def test_losses_move_as_their_gradients_say(name):
    """Along a direction, with the same formulas in 64 bits from bf16 parameters: the gradient passes through bf16
    tensors (four at most, each within 2^-8 of its value), so a slope is within 2^-6 of the sum of its terms' sizes."""
    n = 24
    block = decoder_block.DecoderBlock(max_tokens=n, seed=5)
    residual, previous, positions, o_target, y_target = _inputs(block, n, 6)
    _, _, s, g = block.train_step(residual, previous, positions, o_target, y_target)
    names = ("qkv", "qkv_bias", "q_norm", "k_norm", "out", "dense_up", "dense_bias", "dense_down")
    p = {k: getattr(block, k).to(D) for k in names}
    rest = s["y"].to(D) - s["d"].to(D)
    v = torch.randn(p[name].shape, generator=torch.Generator().manual_seed(7)).cuda().to(D)

    def losses(step):
        q = dict(p)
        q[name] = p[name] + step * v
        rows = s["x1"].to(D) @ q["qkv"].t() + q["qkv_bias"]
        a, b, c = block.split(rows)
        a, b = _qk(block, a, q["q_norm"], positions)[0], _qk(block, b, q["k_norm"], positions)[0]
        per = block.heads // block.kv_heads
        b, c = b.repeat_interleave(per, 1), c.repeat_interleave(per, 1)
        w = torch.einsum("qhd,khd->hqk", a, b) * block.D ** -0.5
        w = w.masked_fill(torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), -torch.inf).softmax(-1)
        o = torch.einsum("hqk,khd->qhd", w, c).flatten(1) @ q["out"].t()
        h = (s["x2"].to(D) @ q["dense_up"].t() + q["dense_bias"]).clamp(min=0).square()
        y = s["r2"].to(D) + h @ q["dense_down"].t() + rest
        return 0.5 / n * ((o - o_target).square().sum() + (y - y_target).square().sum())

    eps = 1e-5
    slope = float((losses(eps) - losses(-eps)) / (2 * eps))
    terms = g[name].to(D) * v
    assert abs(float(terms.sum()) - slope) <= 2.0 ** -6 * float(terms.abs().sum()), (float(terms.sum()), slope)
    block.close()


def test_the_example_runs(monkeypatch, capsys):
    monkeypatch.setattr(sys, "argv", ["decoder_block.py", "--tokens", "16", "--steps", "2"])
    decoder_block.main()
    assert "step 1" in capsys.readouterr().out
