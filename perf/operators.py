"""Performance cases of the operators around the MoE layer: the norms before and after a block, the router's balance loss
and backward pass, and the low-rank adapters beside a shared projection.

Each case names an operator and its sizes.  ``prepare`` makes what a program has in hand before the call, ``run`` is one
pass (the plain form in elementary torch operations in 32 bits, or the library's calls where ``own`` is set), ``exact``
the same result from the definition in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4}


# ------------------------------------------------------------------ cases

def _norm(name, op, n, hidden, residual, branch, gate, sigmoid, post, param="bf16", offset=0.0, alpha=1.0, beta=1.0):
    return {"name": name, "op": op, "n": n, "hidden": hidden, "residual": residual, "branch": branch, "gate": gate,
            "sigmoid": sigmoid, "post": post, "param": param, "offset": offset, "alpha": alpha, "beta": beta}


def _router(name, op, n, experts, k, seqs, masked, sigma):
    return {"name": name, "op": op, "n": n, "experts": experts, "k": k, "seqs": seqs, "masked": masked, "sigma": sigma}


def _lora(name, n, inp, out, adapters, rank, requests, y, o, mixed):
    return {"name": name, "op": "lora", "n": n, "in": inp, "out": out, "adapters": adapters, "rank": rank,
            "requests": requests, "y": y, "o": o, "mixed": mixed}


def listed():
    return [
        # one decoded token between two blocks: the post-norm of the MoE output, its per-channel gate, the scaled
        # residual and the next block's pre-norm in one call; latency
        _norm("norm-1", "norm", 1, 2688, "bf16", "bf16", "channel", False, True, beta=0.25),
        # the long prefill of the 4096-wide configuration with an fp32 residual stream and a sigmoid gate per token
        _norm("norm-16384", "norm", 16384, 4096, "fp32", "bf16", "token", True, True, param="fp32"),
        # a short, odd training batch with a gate of its own for every element and an odd width
        _norm("norm-bwd-61", "norm_bwd", 61, 1000, "fp32", "fp32", "full", False, True, param="fp32", offset=1.0),
        # the training counterpart of the 4314-token prefill
        _norm("norm-bwd-4314", "norm_bwd", 4314, 2688, "bf16", "bf16", "channel", False, True, beta=0.5),
        # a small router, a few tokens, one sequence
        _router("balance-33", "balance", 33, 40, 3, 1, 0.0, 0.5),
        # a packed training batch: sequences of uneven lengths, padding tokens masked, skewed routing
        _router("balance-16384", "balance", 16384, 128, 8, 7, 0.1, 2.0),
        # the router's backward pass for the 4314-token batch
        _router("router-bwd-4314", "router_bwd", 4314, 128, 6, 3, 0.05, 1.5),
        # and for a long batch over 512 experts
        _router("router-bwd-16384", "router_bwd", 16384, 512, 8, 12, 0.1, 2.0),
        # one decoded token of one request with an adapter; latency
        _lora("lora-1", 1, 2688, 1856, 8, 16, 1, "bf16", "bf16", False),
        # a decode batch, every token another request, adapters of different ranks, some requests without one
        _lora("lora-32", 32, 2688, 1856, 16, 32, 32, "fp32", "bf16", True),
        # a prefill of a few requests on the shared projection's fp32 result
        _lora("lora-4314", 4314, 2688, 1856, 8, 16, 9, "fp32", "fp32", False),
        # the long prefill with larger ranks
        _lora("lora-16384", 16384, 4096, 2048, 12, 64, 24, "bf16", "bf16", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "norm_bwd", "balance", "router_bwd", "lora", "lora", "lora"])
    if op in ("norm", "norm_bwd"):
        hidden = 8 * _log(rng, 32, 1024)
        most = 16384 * 4096 if op == "norm" else 4314 * 2688
        n = _log(rng, 1, min(16384, most // hidden))
        c = _norm("", op, n, hidden, rng.choice(["bf16", "fp32"]), rng.choice(["bf16", "fp32"]),
                  rng.choice(["none", "channel", "token", "full"]), rng.random() < 0.5, rng.random() < 0.75,
                  rng.choice(["bf16", "fp32"]), rng.choice([0.0, 1.0]), rng.choice([1.0, 1.5]), rng.choice([1.0, 0.25]))
        wide = 2.0 if "fp32" in (c["residual"], c["branch"]) else 1.0
        if c["gate"] == "full":
            wide *= 1.4
        c["n"] = max(1, min(n, int(most / hidden / wide)))
        c["sigmoid"] = c["sigmoid"] and c["gate"] != "none"
    elif op in ("balance", "router_bwd"):
        experts = _log(rng, 8, 1024)
        k = rng.randint(1, min(8, experts))
        n = _log(rng, 1, min(16384, 16384 * (128 if op == "balance" else 512) // experts))
        c = _router("", op, n, experts, k, min(n, rng.choice([1, 1, 2, 5, 16])), rng.choice([0.0, 0.1, 0.4]),
                    rng.choice([0.0, 1.5]))
    else:
        inp, out = 8 * _log(rng, 32, 512), 8 * _log(rng, 32, 512)
        y = rng.choice(["bf16", "fp32"])
        o = "bf16" if y == "bf16" else rng.choice(["bf16", "fp32"])
        moved = 2 * inp + (BYTES[y] + BYTES[o]) * out  # bytes a token; the longest listed case moves 16384 x 16384
        n = _log(rng, 1, min(16384, 16384 * 6144 // (inp + out), 16384 * 16384 // moved))
        decode = n <= 256 and rng.random() < 0.7
        rank = rng.choice([8, 16, 16, 32, 64])
        c = _lora("", n, inp, out, rng.randint(1, min(24, 768 // rank)), rank,
                  n if decode else min(n, rng.randint(1, 24)), y, o, rng.random() < 0.5)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _lengths(total, parts, g):
    """Boundaries of `parts` uneven runs of `total` things, int32 [parts + 1] on the device (a run may be empty)."""
    if parts >= total:
        return torch.arange(parts + 1, dtype=torch.int32, device=DEV).clamp_(max=total)
    cuts = torch.rand(parts - 1, generator=g, device=DEV).mul_(total).to(torch.int32).sort().values
    end = torch.tensor([0, total], dtype=torch.int32, device=DEV)
    return torch.cat([end[:1], cuts, end[1:]]).contiguous()


def _prepare_norm(c, g):
    n, H = c["n"], c["hidden"]
    res, act, par = TYPES[c["residual"]], TYPES[c["branch"]], TYPES[c["param"]]
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    s = {"case": c, "residual": (2.0 * randn(n, H)).to(res), "branch": (randn(n, H) * 0.5).to(act)}
    s["pre"] = (randn(H) * 0.1 + 1.0 - c["offset"]).to(par)
    s["post"] = (randn(H) * 0.1 + 1.0 - c["offset"]).to(par) if c["post"] else None
    shape, kind = {"none": (None, None), "channel": ((H,), par), "token": ((n, 1), torch.float32),
                   "full": ((n, H), act)}[c["gate"]]
    s["gate"] = None if shape is None else randn(*shape).to(kind)
    if c["op"] == "norm":
        s["residual_out"] = torch.empty(n, H, dtype=res, device=DEV)
        s["x"] = torch.empty(n, H, dtype=torch.bfloat16, device=DEV)
        s["rstd_post"] = torch.empty(n, device=DEV) if c["post"] else None
        s["rstd_pre"] = torch.empty(n, device=DEV)
        return s
    # the backward pass has the forward's residual_out and row statistics, and the gradients of what it returned
    mean = lambda t: torch.rsqrt(t.double().square().mean(1) + EPS).float()  # noqa: E731
    s["rstd_pre"] = mean(s["residual"])
    s["rstd_post"] = mean(s["branch"]) if c["post"] else None
    s["d_residual_out"] = randn(n, H).to(res)
    s["d_x"] = randn(n, H).to(torch.bfloat16)
    s["d_residual"] = torch.empty(n, H, dtype=res, device=DEV)
    s["d_branch"] = torch.empty(n, H, dtype=act, device=DEV)
    s["d_gate"] = None if s["gate"] is None else torch.empty(
        s["gate"].shape, dtype=act if c["gate"] == "full" else torch.float32, device=DEV)
    s["d_pre"] = torch.empty(H, device=DEV)
    s["d_post"] = torch.empty(H, device=DEV) if c["post"] else None
    return s


def _prepare_router(c, g):
    n, E, k, S = c["n"], c["experts"], c["k"], c["seqs"]
    s = {"case": c, "coef": 0.01, "logits": torch.randn(n, E, generator=g, device=DEV)}
    s["bias"] = torch.randn(E, generator=g, device=DEV) * c["sigma"] if c["sigma"] else None
    z = s["logits"] if s["bias"] is None else s["logits"] + s["bias"]
    top = z.topk(k, dim=1)
    s["ids"] = top.indices.to(torch.int32)
    s["weights"] = torch.softmax(top.values, 1)
    s["mask"] = (torch.rand(n, generator=g, device=DEV) >= c["masked"]) if c["masked"] else None
    s["seq_offsets"] = _lengths(n, S, g) if S > 1 else None
    s["loss"] = torch.empty(1, device=DEV)
    s["counts"] = torch.empty(S, E, dtype=torch.int32, device=DEV)
    s["prob_sums"] = torch.empty(S, E, device=DEV)
    s["tokens"] = torch.empty(S + 1, dtype=torch.int32, device=DEV)
    if c["op"] == "router_bwd":
        kept = torch.ones(n, dtype=torch.bool, device=DEV) if s["mask"] is None else s["mask"]
        seq = _sequence(s).long()
        s["counts"].zero_()
        s["counts"].view(-1).index_add_(0, (seq[:, None] * E + s["ids"].long()).view(-1),
                                        kept[:, None].expand(n, k).reshape(-1).to(torch.int32))
        s["tokens"].zero_()
        s["tokens"].index_add_(0, seq, kept.to(torch.int32))
        s["tokens"][S] = s["tokens"][:S].sum().to(torch.int32)
        s["d_weights"] = torch.randn(n, k, generator=g, device=DEV) * (0.01 / n)  # of the size of the loss term
        s["d_loss"] = torch.rand(1, generator=g, device=DEV) + 0.5
        s["d_logits"] = torch.empty(n, E, device=DEV)
        s["d_bias"] = torch.empty(E, device=DEV)
    return s


def _prepare_lora(c, g):
    n, inp, out, L, R = c["n"], c["in"], c["out"], c["adapters"], c["rank"]
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    s = {"case": c, "x": randn(n, inp).to(torch.bfloat16)}
    s["a"] = (randn(L, R, inp) / math.sqrt(inp)).to(torch.bfloat16)
    s["b"] = (randn(L, out, R) / math.sqrt(R)).to(torch.bfloat16)
    s["scale"] = torch.rand(L, generator=g, device=DEV) + 0.5
    s["ranks"] = None
    if c["mixed"]:  # ranks of 8, 16, ... up to the bank's
        s["ranks"] = (8 * (1 + torch.floor(torch.rand(L, generator=g, device=DEV) * (R // 8)))).to(torch.int32)
    # requests without an adapter: about one in eight, where there are several
    per = torch.randint(0, L, (c["requests"],), generator=g, device=DEV, dtype=torch.int32)
    if c["requests"] > 1:
        per = torch.where(torch.rand(c["requests"], generator=g, device=DEV) < 0.125, -1, per).to(torch.int32)
    runs = _lengths(n, c["requests"], g)
    s["ids"] = per[torch.searchsorted(runs[1:].contiguous(), torch.arange(n, dtype=torch.int32, device=DEV),
                                      right=True)].contiguous()
    s["y"] = randn(n, out).to(TYPES[c["y"]])
    s["out"] = torch.empty(n, out, dtype=TYPES[c["o"]], device=DEV)
    return s


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] in ("norm", "norm_bwd"):
        return _prepare_norm(case, g)
    if case["op"] in ("balance", "router_bwd"):
        return _prepare_router(case, g)
    return _prepare_lora(case, g)


# ------------------------------------------------------------------ plain forms

def _sequence(s):
    """Each token's sequence."""
    n = s["logits"].shape[0]
    if s["seq_offsets"] is None:
        return torch.zeros(n, dtype=torch.int32, device=DEV)
    at = torch.arange(n, dtype=torch.int32, device=DEV)
    return torch.searchsorted(s["seq_offsets"][1:].contiguous(), at, right=True).to(torch.int32)


def _plain_norm(s):
    c = s["case"]
    y, post = s["branch"].float(), s["post"]
    rstd_post = None
    if post is not None:
        rstd_post = torch.rsqrt((y * y).mean(1) + EPS)
        y = y * rstd_post[:, None] * (post.float() + c["offset"])
    if s["gate"] is not None:
        gate = s["gate"].float()
        y = y * (1.0 / (1.0 + torch.exp(-gate)) if c["sigmoid"] else gate)
    u = c["alpha"] * s["residual"].float() + c["beta"] * y
    rstd_pre = torch.rsqrt((u * u).mean(1) + EPS)
    x = u * rstd_pre[:, None] * (s["pre"].float() + c["offset"])
    return {"residual_out": u.to(s["residual"].dtype), "x": x.to(torch.bfloat16), "rstd_post": rstd_post,
            "rstd_pre": rstd_pre}


def _plain_norm_bwd(s):
    c = s["case"]
    u, dx, ru = s["residual"].float(), s["d_x"].float(), s["rstd_pre"][:, None]
    dxw = dx * (s["pre"].float() + c["offset"])
    xhat = u * ru
    d_pre = (dx * xhat).sum(0)
    G = s["d_residual_out"].float() + ru * (dxw - xhat * (dxw * xhat).mean(1, keepdim=True))
    y = s["branch"].float()
    yhat = y if s["post"] is None else y * s["rstd_post"][:, None]
    w = 1.0 if s["post"] is None else s["post"].float() + c["offset"]
    gate, d_gate = 1.0, None
    if s["gate"] is not None:
        raw = s["gate"].float()
        gate = 1.0 / (1.0 + torch.exp(-raw)) if c["sigmoid"] else raw
        d_gate = c["beta"] * yhat * w * G
        if c["gate"] == "channel":
            d_gate = d_gate.sum(0)
        elif c["gate"] == "token":
            d_gate = d_gate.sum(1, keepdim=True)
        if c["sigmoid"]:
            d_gate = d_gate * gate * (1.0 - gate)
        d_gate = d_gate.to(s["d_gate"].dtype)
    dz = c["beta"] * gate * G
    d_post = None
    dy = dz
    if s["post"] is not None:
        d_post = (dz * yhat).sum(0)
        dzw = dz * w
        dy = s["rstd_post"][:, None] * (dzw - yhat * (dzw * yhat).mean(1, keepdim=True))
    return {"d_residual": (c["alpha"] * G).to(s["residual"].dtype), "d_branch": dy.to(s["branch"].dtype),
            "d_gate": d_gate, "d_post": d_post, "d_pre": d_pre}


def _softmax(s):
    z = s["logits"] if s["bias"] is None else s["logits"] + s["bias"]
    e = torch.exp(z - z.max(1, keepdim=True).values)
    return e / e.sum(1, keepdim=True)


def _plain_balance(s):
    c = s["case"]
    n, E, S, k = c["n"], c["experts"], c["seqs"], c["k"]
    member = (_sequence(s)[None, :] == torch.arange(S, device=DEV)[:, None]).float()  # [S][n]
    if s["mask"] is not None:
        member = member * s["mask"].float()
    picks = (s["ids"][:, :, None] == torch.arange(E, dtype=torch.int32, device=DEV)).sum(1).float()  # [n][E]
    counts, sums, tokens = member @ picks, member @ _softmax(s), member.sum(1)
    total = tokens.sum()
    per = (counts * sums).sum(1) / tokens.clamp(min=1.0)
    loss = s["coef"] * E / (total.clamp(min=1.0) * k) * per.sum()
    return {"loss": loss.reshape(1), "counts": counts.to(torch.int32), "prob_sums": sums,
            "tokens": torch.cat([tokens, total[None]]).to(torch.int32)}


def _plain_router_bwd(s):
    c = s["case"]
    E, S, k = c["experts"], c["seqs"], c["k"]
    seq = _sequence(s).long()
    per = s["counts"].float() / s["tokens"][:S, None].float().clamp(min=1.0)
    g = (s["d_loss"] * (s["coef"] * E) / (s["tokens"][S].float().clamp(min=1.0) * k)) * per[seq]  # [n][E]
    if s["mask"] is not None:
        g = g * s["mask"].float()[:, None]
    p = _softmax(s)
    d = p * (g - (g * p).sum(1, keepdim=True))
    w, dw = s["weights"], s["d_weights"]
    dz = w * (dw - (w * dw).sum(1, keepdim=True))
    d = d.scatter_add(1, s["ids"].long(), dz)
    return {"d_logits": d, "d_bias": d.sum(0)}


def _plain_lora(s):
    c = s["case"]
    n, L, R, inp, out = c["n"], c["adapters"], c["rank"], c["in"], c["out"]
    x, ids = s["x"].float(), s["ids"].long()
    live = (ids >= 0)
    at = ids.clamp(min=0)
    scale = s["scale"][at] * live.float()
    ranks = torch.full((L,), R, dtype=torch.int32, device=DEV) if s["ranks"] is None else s["ranks"]
    keep = torch.arange(R, device=DEV)[None, :] < ranks[:, None]  # [L][R]
    if n <= L:  # few tokens: each takes its own adapter
        v = torch.matmul(s["a"][at].float(), x[:, :, None])[:, :, 0] * keep[at].float()
        delta = torch.matmul(s["b"][at].float(), v[:, :, None])[:, :, 0]
    else:  # every adapter's columns side by side, each token keeps those of its own
        v = x @ s["a"].float().reshape(L * R, inp).t()
        mine = (at[:, None, None] == torch.arange(L, device=DEV)[None, :, None]) & keep[None]
        delta = (v * mine.reshape(n, L * R).float()) @ s["b"].float().permute(0, 2, 1).reshape(L * R, out)
    return {"out": (s["y"].float() + scale[:, None] * delta).to(s["out"].dtype)}


_PLAIN = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "balance": _plain_balance, "router_bwd": _plain_router_bwd,
          "lora": _plain_lora}


# ------------------------------------------------------------------ the library's calls

def _own_norm(s):
    from nvfp4_quantized_moe_topk_gb300 import api

    c = s["case"]
    api.block_norm(s["residual"], s["branch"], s["gate"], s["post"], s["pre"], s["residual_out"], s["x"],
                   s["rstd_post"], s["rstd_pre"], eps=EPS, residual_scale=c["alpha"], branch_scale=c["beta"],
                   weight_offset=c["offset"], gate_sigmoid=c["sigmoid"])
    return {"residual_out": s["residual_out"], "x": s["x"], "rstd_post": s["rstd_post"], "rstd_pre": s["rstd_pre"]}


def _own_norm_bwd(s):
    from nvfp4_quantized_moe_topk_gb300 import api

    c = s["case"]
    if "workspace" not in s:
        s["workspace"] = api.block_norm_workspace(c["n"], c["hidden"])
    api.block_norm_backward(s["d_residual_out"], s["d_x"], s["residual"], s["branch"], s["gate"], s["post"], s["pre"],
                            s["rstd_post"], s["rstd_pre"], s["d_residual"], s["d_branch"], s["d_gate"], s["d_post"],
                            s["d_pre"], residual_scale=c["alpha"], branch_scale=c["beta"], weight_offset=c["offset"],
                            gate_sigmoid=c["sigmoid"], workspace=s["workspace"])
    return {"d_residual": s["d_residual"], "d_branch": s["d_branch"], "d_gate": s["d_gate"], "d_post": s["d_post"],
            "d_pre": s["d_pre"]}


def _own_balance(s):
    from nvfp4_quantized_moe_topk_gb300 import api

    c = s["case"]
    if "workspace" not in s:
        s["workspace"] = api.router_workspace(c["n"], c["experts"], c["seqs"])
    api.balance_loss(s["logits"], s["bias"], s["ids"], s["loss"], s["counts"], s["prob_sums"], s["tokens"],
                     coef=s["coef"], mask=s["mask"], seq_offsets=s["seq_offsets"], workspace=s["workspace"])
    return {"loss": s["loss"], "counts": s["counts"], "prob_sums": s["prob_sums"], "tokens": s["tokens"]}


def _own_router_bwd(s):
    from nvfp4_quantized_moe_topk_gb300 import api

    c = s["case"]
    if "workspace" not in s:
        s["workspace"] = api.router_workspace(c["n"], c["experts"], c["seqs"])
    api.router_backward(s["logits"], s["bias"], s["ids"], s["weights"], s["d_weights"], s["counts"], s["tokens"],
                        s["d_logits"], s["d_bias"], d_loss=s["d_loss"], coef=s["coef"], mask=s["mask"],
                        seq_offsets=s["seq_offsets"], workspace=s["workspace"])
    return {"d_logits": s["d_logits"], "d_bias": s["d_bias"]}


def _own_lora(s):
    from nvfp4_quantized_moe_topk_gb300 import api

    if "workspace" not in s:
        s["workspace"] = api.lora_workspace(s["x"].shape[0], s["a"].shape[0])
    api.lora_apply(s["x"], s["ids"], s["a"], s["b"], s["y"], s["out"], scale=s["scale"], ranks=s["ranks"],
                   workspace=s["workspace"])
    return {"out": s["out"]}


_OWN = {"norm": _own_norm, "norm_bwd": _own_norm_bwd, "balance": _own_balance, "router_bwd": _own_router_bwd,
        "lora": _own_lora}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    n = c["n"]
    if c["op"] in ("norm", "norm_bwd"):
        H, res, act, par = c["hidden"], BYTES[c["residual"]], BYTES[c["branch"]], BYTES[c["param"]]
        gate = {"none": 0, "channel": H * par, "token": 4 * n, "full": n * H * act}[c["gate"]]
        rows = 4 * n * (2 if c["post"] else 1)
        vec = H * (2 if c["post"] else 1)
        if c["op"] == "norm":
            return {"bytes": n * H * (2 * res + act + 2) + gate + rows + vec * par, "flops": 12 * n * H}
        d_gate = {"none": 0, "channel": 4 * H, "token": 4 * n, "full": n * H * act}[c["gate"]]
        return {"bytes": n * H * (3 * res + 2 * act + 2) + gate + d_gate + rows + vec * (par + 4), "flops": 30 * n * H}
    if c["op"] in ("balance", "router_bwd"):
        E, k, S = c["experts"], c["k"], c["seqs"]
        bias, mask, seq = (4 * E if c["sigma"] else 0), (n if c["masked"] else 0), (4 * (S + 1) if S > 1 else 0)
        if c["op"] == "balance":
            return {"bytes": 4 * n * (E + k) + bias + mask + seq + 8 * S * E + 4 * (S + 2), "flops": 6 * n * E}
        return {"bytes": 8 * n * E + 12 * n * k + bias + mask + seq + 4 * S * E + 4 * (S + 2) + 4 * E,
                "flops": 10 * n * E}
    inp, out, R = c["in"], c["out"], c["rank"]
    used = min(c["adapters"], c["requests"])
    rank = (R + 8) / 2 if c["mixed"] else R  # the mean of the drawn ranks
    return {"bytes": int(n * (2 * inp + (BYTES[c["y"]] + BYTES[c["o"]]) * out + 4) + used * rank * (inp + out) * 2),
            "flops": int(2 * n * rank * (inp + out))}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_norm(c, s):
    D = torch.float64
    y = s["branch"].to(D)
    rp = None
    if s["post"] is not None:
        rp = (y.pow(2).mean(-1) + EPS).pow(-0.5)
        y = torch.einsum("th,t,h->th", y, rp, s["post"].to(D) + c["offset"])
    if s["gate"] is not None:
        q = s["gate"].to(D)
        y = y * (q.sigmoid() if c["sigmoid"] else q)
    u = s["residual"].to(D).mul(c["alpha"]).add(y, alpha=c["beta"])
    ru = (u.pow(2).mean(-1) + EPS).pow(-0.5)
    return {"residual_out": u, "x": torch.einsum("th,t,h->th", u, ru, s["pre"].to(D) + c["offset"]), "rstd_post": rp,
            "rstd_pre": ru}


def _exact_norm_bwd(c, s):
    """By automatic differentiation of the definition: d(sum u * d_residual_out + sum x * d_x), u the stored residual
    (a variable of its own for the gradient that reaches it, then passed on to the branch)."""
    D = torch.float64
    leaf = lambda t: None if t is None else t.to(D).requires_grad_(True)  # noqa: E731
    u, pre = leaf(s["residual"]), leaf(s["pre"])
    x = u * (u.pow(2).mean(-1, keepdim=True) + EPS).pow(-0.5) * (pre + c["offset"])
    G, d_pre = torch.autograd.grad([x], [u, pre], [s["d_x"].to(D)])
    G = G + s["d_residual_out"].to(D)
    y, gate, post = leaf(s["branch"]), leaf(s["gate"]), leaf(s["post"])
    z = y
    if post is not None:
        z = z * (y.pow(2).mean(-1, keepdim=True) + EPS).pow(-0.5) * (post + c["offset"])
    if gate is not None:
        z = z * (gate.sigmoid() if c["sigmoid"] else gate)
    want = [t for t in (y, gate, post) if t is not None]
    got = dict(zip([id(t) for t in want], torch.autograd.grad([c["beta"] * z], want, [G])))
    return {"d_residual": c["alpha"] * G, "d_branch": got[id(y)], "d_gate": got.get(id(gate)),
            "d_post": got.get(id(post)), "d_pre": d_pre}


def _exact_router(c, s):
    """The loss over each sequence's own rows, and its gradient and the weights' by automatic differentiation."""
    D = torch.float64
    n, E, S, k = c["n"], c["experts"], c["seqs"], c["k"]
    z = s["logits"] if s["bias"] is None else s["logits"] + s["bias"]  # one addition in 32 bits, as defined
    z = z.to(D).requires_grad_(True)
    p = torch.softmax(z, 1)
    kept = torch.ones(n, dtype=torch.bool, device=DEV) if s["mask"] is None else s["mask"]
    ends = [0, n] if s["seq_offsets"] is None else s["seq_offsets"].tolist()
    total = int(kept.sum())
    loss, sums = z.new_zeros(()), []
    for i in range(S):
        rows = slice(ends[i], ends[i + 1])
        mine = p[rows][kept[rows]]
        picks = torch.bincount(s["ids"][rows][kept[rows]].reshape(-1).long(), minlength=E).to(D)
        sums.append(mine.sum(0))
        if mine.shape[0]:
            f, P = picks / (mine.shape[0] * k), mine.mean(0)
            loss = loss + (mine.shape[0] / total) * E * (f * P).sum()
    loss = s["coef"] * loss
    if c["op"] == "balance":
        return {"loss": loss.detach().reshape(1), "counts": None, "prob_sums": torch.stack(sums).detach(),
                "tokens": None}
    w = torch.softmax(z.gather(1, s["ids"].long()), 1)
    scalar = loss * float(s["d_loss"]) + (w * s["d_weights"].to(D)).sum()
    d, = torch.autograd.grad([scalar], [z])
    return {"d_logits": d, "d_bias": d.sum(0)}


def _exact_lora(c, s):
    D = torch.float64
    out = s["y"].to(D)
    ranks = [c["rank"]] * c["adapters"] if s["ranks"] is None else s["ranks"].tolist()
    for a in range(c["adapters"]):
        rows = (s["ids"] == a).nonzero()[:, 0]
        if rows.numel():
            r = ranks[a]
            v = s["x"][rows].to(D) @ s["a"][a, :r].to(D).T
            out[rows] += float(s["scale"][a]) * (v @ s["b"][a, :, :r].to(D).T)
    return {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        return _exact_norm(case, s)
    if op == "norm_bwd":
        return _exact_norm_bwd(case, s)
    if op in ("balance", "router_bwd"):
        return _exact_router(case, s)
    return _exact_lora(case, s)
