"""Performance cases of the operators on the way into and through a block: the projections (a matrix product with bias,
activation and residual in its epilogue) with their backward pass, the norms of queries and keys with the rotation of
their positions, forward and backward, and the whole MoE layer (router, shared and routed experts) for a few tokens.

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

def _linear(name, op, n, inp, out, act, bias, residual, o, z="none", w="bf16"):
    """residual, z: their type or "none"; o: the type of out, or of the gradients d_out and d_x; w: of d_weight."""
    return {"name": name, "op": op, "n": n, "in": inp, "out": out, "act": act, "bias": bias, "residual": residual,
            "o": o, "z": z, "w": w}


def _qk(name, op, n, heads, kv_heads, dim, rot, axes, norm, dtype, interleaved=False, mixed_axes=False, fused=True,
        offset=0.0, base=10000.0, far=4096):
    """rot: rotated dimensions of a head; interleaved: pairs side by side; fused: q and k are views into one
    projection's rows; far: positions reach so far."""
    return {"name": name, "op": op, "n": n, "heads": heads, "kv_heads": kv_heads, "dim": dim, "rot": rot, "axes": axes,
            "norm": norm, "dtype": dtype, "interleaved": interleaved, "mixed_axes": mixed_axes, "fused": fused,
            "offset": offset, "base": base, "far": far}


def _layer(name, n, hidden, inter, experts, k, shared, gated, router, residual):
    """experts: routed ones; shared: experts that every token takes; router: the type of its weight."""
    return {"name": name, "op": "layer", "n": n, "hidden": hidden, "inter": inter, "experts": experts, "k": k,
            "shared": shared, "gated": gated, "router": router, "residual": residual}


def listed():
    return [
        # one decoded token through the projection to queries, keys and values (32 and 2 x 2 heads of 128); latency
        _linear("linear-1", "linear", 1, 2688, 4608, "none", True, "none", "bf16"),
        # a decode batch of odd sizes through a small projection onto an fp32 residual stream
        _linear("linear-33", "linear", 33, 1000, 520, "gelu_tanh", True, "fp32", "fp32"),
        # the attention's output projection of the 4314-token prefill onto the residual
        _linear("linear-4314", "linear", 4314, 4096, 2688, "none", False, "bf16", "bf16"),
        # a dense feed-forward's first product in training: long batch, activation, its argument kept for the backward
        _linear("linear-16384", "linear", 16384, 4096, 8192, "relu2", True, "none", "bf16", z="bf16"),
        # the backward pass of a short, odd batch, gradients in 32 bits
        _linear("linear-bwd-61", "linear_bwd", 61, 1000, 520, "silu", True, "none", "fp32", z="fp32", w="fp32"),
        # the training counterpart of the 4314-token batch's projection to queries, keys and values
        _linear("linear-bwd-4314", "linear_bwd", 4314, 2688, 4608, "none", True, "none", "bf16", w="fp32"),
        # one decoded token's queries and keys, far into its context; latency
        _qk("qk-1", "qk", 1, 32, 2, 128, 128, 1, True, "bf16", base=1000000.0, far=131072),
        # a long prefill of text and images: three axes of positions
        _qk("qk-16384", "qk", 16384, 32, 8, 128, 128, 3, True, "bf16", mixed_axes=True, base=1000000.0),
        # a short, odd training batch: few heads, part of an odd head rotated, pairs side by side, fp32
        _qk("qk-bwd-515", "qk_bwd", 515, 5, 1, 80, 32, 2, True, "fp32", interleaved=True, fused=False, offset=1.0),
        # the training counterpart of the 4314-token prefill
        _qk("qk-bwd-4314", "qk_bwd", 4314, 32, 2, 128, 128, 1, True, "bf16"),
        # one decoded token through the whole MoE layer: router, shared expert, six of 128 experts; latency
        _layer("layer-1", 1, 2688, 1856, 128, 6, 1, False, "bf16", "own"),
        # a decode batch with a shared expert of twice the width (two parts), gated, router weight in fp32
        _layer("layer-32", 32, 2688, 1856, 128, 6, 2, True, "fp32", "none"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_bwd", "linear_bwd", "qk", "qk", "qk_bwd", "qk_bwd", "layer", "layer"])
    if op in ("linear", "linear_bwd"):
        inp, out = 8 * _log(rng, 16, 1024), 8 * _log(rng, 16, 1024)
        most = 16384 * 4096 * 8192 // (1 if op == "linear" else 3)
        n = _log(rng, 1, min(16384, max(1, most // (inp * out))))
        act = rng.choice(["none", "none", "relu2", "silu", "gelu_tanh"])
        o = rng.choice(["bf16", "bf16", "fp32"])
        if op == "linear":
            c = _linear("", op, n, inp, out, act, rng.random() < 0.5, rng.choice(["none", "bf16", "fp32"]), o,
                        rng.choice(["none", "bf16", "fp32"]))
        else:
            c = _linear("", op, n, inp, out, act, rng.random() < 0.5, "none", o,
                        "none" if act == "none" else rng.choice(["bf16", "fp32"]), rng.choice(["bf16", "fp32"]))
    elif op in ("qk", "qk_bwd"):
        kv = rng.choice([1, 2, 4, 5, 8])
        heads = kv * rng.choice([1, 2, 5, 8])
        dim = rng.choice([32, 64, 80, 96, 128, 128, 192, 256])
        rot = 16 * rng.randint(1, dim // 16) if rng.random() < 0.4 else dim
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        most = 16384 * 40 * 128 if op == "qk" else 4314 * 36 * 128  # elements that are read and written
        n = _log(rng, 1, min(16384, max(1, most * 2 // (BYTES[dtype] * (heads + kv) * dim))))
        c = _qk("", op, n, heads, kv, dim, rot, rng.randint(1, 4), rng.random() < 0.8, dtype, rng.random() < 0.3,
                rng.random() < 0.5, rng.random() < 0.7, rng.choice([0.0, 1.0]), rng.choice([10000.0, 1000000.0]),
                rng.choice([512, 4096, 131072, 1048576]))
        c["axes"] = min(c["axes"], rot // 2)
    else:
        hidden, inter = 64 * _log(rng, 4, 42), 64 * _log(rng, 2, 29)
        experts = _log(rng, 8, 128)
        c = _layer("", _log(rng, 1, 32), hidden, inter, experts, rng.randint(1, min(6, experts)), rng.randint(0, 2),
                   rng.random() < 0.5, rng.choice(["bf16", "fp32"]), rng.choice(["none", "own"]))
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _prepare_linear(c, g):
    n, inp, out = c["n"], c["in"], c["out"]
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    s = {"case": c, "x": randn(n, inp).to(torch.bfloat16), "w": (randn(out, inp) / math.sqrt(inp)).to(torch.bfloat16)}
    if c["op"] == "linear":
        s["bias"] = randn(out) * 0.5 if c["bias"] else None
        s["residual"] = None if c["residual"] == "none" else randn(n, out).to(TYPES[c["residual"]])
        s["scale"] = 1.0 if c["residual"] == "none" else 0.5
        s["out"] = torch.empty(n, out, dtype=TYPES[c["o"]], device=DEV)
        s["z"] = None if c["z"] == "none" else torch.empty(n, out, dtype=TYPES[c["z"]], device=DEV)
        return s
    s["z"] = None if c["act"] == "none" else randn(n, out).to(TYPES[c["z"]])
    s["d_out"] = randn(n, out).to(TYPES[c["o"]])
    s["d_x"] = torch.empty(n, inp, dtype=TYPES[c["o"]], device=DEV)
    s["d_w"] = torch.empty(out, inp, dtype=TYPES[c["w"]], device=DEV)
    s["d_bias"] = torch.empty(out, device=DEV) if c["bias"] else None
    return s


def _sections(c):
    """Pairs of each axis: even shares, the first axis takes the rest."""
    pairs, axes = c["rot"] // 2, c["axes"]
    return (pairs - (axes - 1) * (pairs // axes),) + (pairs // axes,) * (axes - 1)


def _prepare_qk(c, g):
    n, H, K, D = c["n"], c["heads"], c["kv_heads"], c["dim"]
    t = TYPES[c["dtype"]]
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731

    def pair():
        if c["fused"]:  # rows of queries, keys and values side by side
            rows = randn(n, (H + 2 * K) * D).to(t)
            return rows[:, : H * D].view(n, H, D), rows[:, H * D: (H + K) * D].view(n, K, D)
        return randn(n, H, D).to(t), randn(n, K, D).to(t)

    s = {"case": c}
    s["q"], s["k"] = pair()
    weight = lambda: (randn(D) * 0.1 + 1.0 - c["offset"]).to(t) if c["norm"] else None  # noqa: E731
    s["q_w"], s["k_w"] = weight(), weight()
    i = torch.arange(c["rot"] // 2, device=DEV, dtype=torch.float64)
    s["inv_freq"] = torch.pow(torch.tensor(c["base"], dtype=torch.float64, device=DEV), -2.0 * i / c["rot"]).float()
    # the first axis runs on through the batch from somewhere in the context, the others over an image's rows and columns
    pos = torch.randint(0, c["far"], (c["axes"], n), generator=g, device=DEV, dtype=torch.int32)
    start = int(torch.randint(0, c["far"], (1,), generator=g, device=DEV))
    pos[0] = start + torch.arange(n, dtype=torch.int32, device=DEV)
    s["positions"] = pos
    s["sections"] = _sections(c)
    if c["op"] == "qk":
        s["q_out"], s["k_out"] = torch.empty(n, H, D, dtype=t, device=DEV), torch.empty(n, K, D, dtype=t, device=DEV)
        return s
    s["d_q_out"], s["d_k_out"] = randn(n, H, D).to(t), randn(n, K, D).to(t)
    s["d_q"], s["d_k"] = torch.empty(n, H, D, dtype=t, device=DEV), torch.empty(n, K, D, dtype=t, device=DEV)
    s["d_q_w"] = torch.empty(D, device=DEV) if c["norm"] else None
    s["d_k_w"] = torch.empty(D, device=DEV) if c["norm"] else None
    return s


def _prepare_layer(c, g):
    n, H, I, E, S = c["n"], c["hidden"], c["inter"], c["experts"], c["shared"]
    rint = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=DEV, dtype=torch.uint8)  # noqa: E731
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    s = {"case": c, "x": randn(n, H).to(torch.bfloat16)}
    # codes of any value, block scales of 1 to 1.875 (e4m3 bytes), globals that keep rows at the size of their inputs
    for name, rows, cols in (("up", I, H), ("down", H, I)) + ((("gate", I, H),) if c["gated"] else ()):
        s[name + "_codes"] = rint(0, 256, E + S, rows, cols // 2)
        s[name + "_scales"] = rint(0x38, 0x40, E + S, rows, cols // 16)
        s[name + "_global"] = (torch.rand(E + S, generator=g, device=DEV) * 0.1 + 0.2) / math.sqrt(cols)
    s["router"] = (randn(E, H) / math.sqrt(H)).to(TYPES[c["router"]])
    s["bias"] = randn(E) * 0.5
    s["residual"] = randn(n, H).to(torch.bfloat16) if c["residual"] == "own" else None
    s["dst"] = torch.empty(n, H, dtype=torch.bfloat16, device=DEV)
    s["ids"] = torch.empty(n, c["k"], dtype=torch.int32, device=DEV)
    s["weights"] = torch.empty(n, c["k"], device=DEV)
    return s


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] in ("linear", "linear_bwd"):
        return _prepare_linear(case, g)
    if case["op"] in ("qk", "qk_bwd"):
        return _prepare_qk(case, g)
    return _prepare_layer(case, g)


# ------------------------------------------------------------------ plain forms

_GELU = math.sqrt(2.0 / math.pi)


def _act(z, act):
    if act == "relu2":
        r = torch.clamp(z, min=0.0)
        return r * r
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu_tanh":
        return z / (1.0 + torch.exp(-2.0 * _GELU * (z + 0.044715 * z * z * z)))  # z/2 (1 + tanh u) = z / (1 + e^-2u)
    return z


def _act_slope(z, act):
    if act == "relu2":
        return 2.0 * torch.clamp(z, min=0.0)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    if act == "gelu_tanh":
        p = 1.0 / (1.0 + torch.exp(-2.0 * _GELU * (z + 0.044715 * z * z * z)))
        return p + z * p * (1.0 - p) * 2.0 * _GELU * (1.0 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _plain_linear(s):
    c = s["case"]
    z = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"]
    out = _act(z, c["act"])
    if s["residual"] is not None:
        out = out + s["scale"] * s["residual"].float()
    return {"out": out.to(s["out"].dtype), "z": None if s["z"] is None else z.to(s["z"].dtype)}


def _plain_linear_bwd(s):
    c = s["case"]
    dz = s["d_out"].float()
    if c["act"] != "none":
        dz = dz * _act_slope(s["z"].float(), c["act"])
    return {"d_x": (dz @ s["w"].float()).to(s["d_x"].dtype), "d_w": (dz.t() @ s["x"].float()).to(s["d_w"].dtype),
            "d_bias": dz.sum(0) if c["bias"] else None}


def _axis_of_pair(c, sections):
    """Which axis's position turns each pair: runs of the sections, or the axes in turn until their sections are full
    and the first axis for the rest."""
    pairs, axes = c["rot"] // 2, c["axes"]
    i = torch.arange(pairs, device=DEV)
    if c["mixed_axes"]:
        turn = i % axes
        share = torch.tensor(sections, device=DEV)[turn]
        return torch.where(i < axes * share, turn, torch.zeros_like(turn))
    ends = torch.tensor(sections, device=DEV).cumsum(0)
    return torch.searchsorted(ends, i, right=True)


def _cos_sin(s):
    c = s["case"]
    at = s["positions"][_axis_of_pair(c, s["sections"])].double().t()  # [n][pairs]
    angle = at * s["inv_freq"].double()
    return torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]


def _halves(x, c):
    """The two members of each pair and what is not rotated."""
    r = x[..., : c["rot"]]
    if c["interleaved"]:
        return r[..., 0::2], r[..., 1::2], x[..., c["rot"]:]
    h = c["rot"] // 2
    return r[..., :h], r[..., h:], x[..., c["rot"]:]


def _join(a, b, rest, c):
    r = torch.stack([a, b], -1).flatten(-2) if c["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([r, rest], -1)


def _plain_qk(s):
    c = s["case"]
    cos, sin = _cos_sin(s)

    def one(h, w):
        y = h.float()
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * (w.float() + c["offset"])
        a, b, rest = _halves(y, c)
        return _join(a * cos - b * sin, b * cos + a * sin, rest, c).to(h.dtype)

    return {"q_out": one(s["q"], s["q_w"]), "k_out": one(s["k"], s["k_w"])}


def _plain_qk_bwd(s):
    c = s["case"]
    cos, sin = _cos_sin(s)

    def one(h, w, d):
        a, b, rest = _halves(d.float(), c)
        dy = _join(a * cos + b * sin, b * cos - a * sin, rest, c)
        if w is None:
            return dy.to(h.dtype), None
        y = h.float()
        r = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS)
        y = y * r
        dyw = dy * (w.float() + c["offset"])
        return (r * (dyw - y * (dyw * y).mean(-1, keepdim=True))).to(h.dtype), (dy * y).sum((0, 1))

    d_q, d_q_w = one(s["q"], s["q_w"], s["d_q_out"])
    d_k, d_k_w = one(s["k"], s["k_w"], s["d_k_out"])
    return {"d_q": d_q, "d_k": d_k, "d_q_w": d_q_w, "d_k_w": d_k_w}


def _e2m1(device):
    half = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=device)
    return torch.cat([half, -half])


def _unpacked(codes, scales):
    """Weights in 32 bits: the low nibble first, a scale for 16 of a row."""
    b = codes.to(torch.int32)
    v = _e2m1(codes.device)[torch.stack([b & 15, b >> 4], -1)].flatten(-2)
    return v * scales.view(torch.float8_e4m3fn).float().repeat_interleave(16, -1)


def _plain_layer(s):
    c = s["case"]
    n, E, S, k = c["n"], c["experts"], c["shared"], c["k"]
    logits = (s["x"].double() @ s["router"].double().t()).float() + s["bias"]  # (64 bits: picks next to one another)
    top = torch.sort(logits, dim=1, descending=True, stable=True)
    ids, z = top.indices[:, :k], top.values[:, :k]
    e = torch.exp(z - z[:, :1])
    weights = e / e.sum(1, keepdim=True)
    every = torch.arange(E, E + S, device=DEV).expand(n, S)
    pick = torch.cat([ids, every], 1).reshape(-1)  # [n (k + S)] experts
    share = torch.cat([weights, torch.ones(n, S, device=DEV)], 1)
    x = s["x"].float().repeat_interleave(k + S, 0)[:, :, None]
    one = lambda name, v: torch.matmul(  # noqa: E731
        _unpacked(s[name + "_codes"][pick], s[name + "_scales"][pick]), v)[:, :, 0] * s[name + "_global"][pick, None]
    h = one("up", x)
    if c["gated"]:
        g = one("gate", x)
        a = g / (1.0 + torch.exp(-g)) * h
    else:
        a = torch.clamp(h, min=0.0)
        a = a * a
    a = a.to(torch.bfloat16).float()  # the layer's own rounding
    y = (one("down", a[:, :, None]).view(n, k + S, -1) * share[:, :, None]).sum(1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"dst": y.to(torch.bfloat16), "ids": ids.to(torch.int32), "weights": weights}


_PLAIN = {"linear": _plain_linear, "linear_bwd": _plain_linear_bwd, "qk": _plain_qk, "qk_bwd": _plain_qk_bwd,
          "layer": _plain_layer}


# ------------------------------------------------------------------ the library's calls

def _own_linear(s):
    from nvfp4_quantized_moe_topk_gb300 import api

    api.linear(s["x"], s["w"], s["out"], s["bias"], s["residual"], s["z"], activation=s["case"]["act"],
               residual_scale=s["scale"])
    return {"out": s["out"], "z": s["z"]}


def _own_linear_bwd(s):
    from nvfp4_quantized_moe_topk_gb300 import api

    c = s["case"]
    if "workspace" not in s:
        s["workspace"] = api.linear_workspace(c["n"], c["in"], c["out"])
    api.linear_backward(s["d_out"], s["x"], s["w"], s["z"], s["d_x"], s["d_w"], s["d_bias"], activation=c["act"],
                        workspace=s["workspace"])
    return {"d_x": s["d_x"], "d_w": s["d_w"], "d_bias": s["d_bias"]}


def _own_qk(s):
    from nvfp4_quantized_moe_topk_gb300 import api

    c = s["case"]
    api.qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], s["positions"], s["inv_freq"], s["q_w"], s["k_w"], eps=EPS,
                     weight_offset=c["offset"], sections=s["sections"], sections_interleaved=c["mixed_axes"],
                     pairs_interleaved=c["interleaved"])
    return {"q_out": s["q_out"], "k_out": s["k_out"]}


def _own_qk_bwd(s):
    from nvfp4_quantized_moe_topk_gb300 import api

    c = s["case"]
    if "workspace" not in s:
        s["workspace"] = api.qk_workspace(c["n"], c["heads"], c["kv_heads"], c["dim"])
    api.qk_norm_rope_backward(s["d_q_out"], s["d_k_out"], s["q"], s["k"], s["d_q"], s["d_k"], s["positions"],
                              s["inv_freq"], s["q_w"], s["k_w"], s["d_q_w"], s["d_k_w"], eps=EPS,
                              weight_offset=c["offset"], sections=s["sections"], sections_interleaved=c["mixed_axes"],
                              pairs_interleaved=c["interleaved"], workspace=s["workspace"])
    return {"d_q": s["d_q"], "d_k": s["d_k"], "d_q_w": s["d_q_w"], "d_k_w": s["d_k_w"]}


def _own_layer(s):
    from nvfp4_quantized_moe_topk_gb300 import api

    c = s["case"]
    if "layer" not in s:
        gate = {"gate_" + p: s["gate_" + p] for p in ("codes", "scales", "global")} if c["gated"] else {}
        s["layer"] = api.MoeLayer(c["hidden"], c["inter"], c["experts"] + c["shared"], c["k"] + c["shared"], c["n"],
                                  s["up_codes"], s["up_scales"], s["down_codes"], s["down_scales"], s["up_global"],
                                  s["down_global"], **gate)
    s["layer"].layer_forward(s["x"], s["router"], s["dst"], s["residual"], s["bias"], shared_experts=c["shared"],
                             topk_ids=s["ids"], topk_weights=s["weights"])
    return {"dst": s["dst"], "ids": s["ids"], "weights": s["weights"]}


_OWN = {"linear": _own_linear, "linear_bwd": _own_linear_bwd, "qk": _own_qk, "qk_bwd": _own_qk_bwd, "layer": _own_layer}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    n = c["n"]
    if c["op"] == "linear":
        i, o = c["in"], c["out"]
        typ = lambda t: 0 if t == "none" else BYTES[t]  # noqa: E731
        return {"bytes": 2 * (n * i + i * o) + n * o * (typ(c["o"]) + typ(c["residual"]) + typ(c["z"])) +
                (4 * o if c["bias"] else 0), "flops": 2 * n * i * o}
    if c["op"] == "linear_bwd":
        i, o = c["in"], c["out"]
        z = BYTES[c["z"]] if c["act"] != "none" else 0
        return {"bytes": n * o * (BYTES[c["o"]] + z) + 2 * (n * i + i * o) + n * i * BYTES[c["o"]] +
                i * o * BYTES[c["w"]] + (4 * o if c["bias"] else 0), "flops": 4 * n * i * o}
    if c["op"] in ("qk", "qk_bwd"):
        e, b = n * (c["heads"] + c["kv_heads"]) * c["dim"], BYTES[c["dtype"]]
        small = 4 * c["axes"] * n + 2 * c["rot"] + (2 * c["dim"] * b if c["norm"] else 0)
        if c["op"] == "qk":
            return {"bytes": 2 * e * b + small, "flops": 9 * e}
        return {"bytes": (3 if c["norm"] else 2) * e * b + small + (8 * c["dim"] if c["norm"] else 0), "flops": 16 * e}
    H, I, E, k, S = c["hidden"], c["inter"], c["experts"], c["k"], c["shared"]
    mats = 3 if c["gated"] else 2
    touched = E * (1.0 - (1.0 - k / E) ** n) + S  # experts that some token takes, on average
    weights = touched * mats * H * I * (0.5 + 1.0 / 16)
    return {"bytes": int(weights + E * H * BYTES[c["router"]] + n * H * (4 + (2 if c["residual"] == "own" else 0)) +
                         8 * n * k), "flops": int(2 * n * (mats * H * I * (k + S) + H * E))}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_linear(c, s):
    D = torch.float64
    z = torch.einsum("ti,oi->to", s["x"].to(D), s["w"].to(D))
    if s["bias"] is not None:
        z += s["bias"].to(D)
    f = {"none": lambda v: v, "relu2": lambda v: v.relu().square(), "silu": lambda v: v * v.sigmoid(),
         "gelu_tanh": lambda v: 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))}[c["act"]]
    out = f(z)
    if s["residual"] is not None:
        out = out.add(s["residual"].to(D), alpha=s["scale"])
    return {"out": out, "z": None if s["z"] is None else z}


def _exact_linear_bwd(c, s):
    """By automatic differentiation of the activation at the kept z, and the products' transposes."""
    D = torch.float64
    d = s["d_out"].to(D)
    if c["act"] != "none":
        z = s["z"].to(D).requires_grad_(True)
        f = {"relu2": lambda v: v.relu().square(), "silu": lambda v: v * v.sigmoid(),
             "gelu_tanh": lambda v: 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))}[c["act"]]
        d, = torch.autograd.grad([f(z)], [z], [d])
    return {"d_x": torch.einsum("to,oi->ti", d, s["w"].to(D)), "d_w": torch.einsum("to,ti->oi", d, s["x"].to(D)),
            "d_bias": d.sum(0) if c["bias"] else None}


def _exact_turns(c, s):
    """exp(i angle) of each token's pairs."""
    sizes, pairs = s["sections"], c["rot"] // 2
    if c["mixed_axes"]:
        axis = [i % c["axes"] if i // c["axes"] < sizes[i % c["axes"]] else 0 for i in range(pairs)]
    else:
        axis = [a for a, size in enumerate(sizes) for _ in range(size)]
    angle = torch.stack([s["positions"][a].double() * s["inv_freq"][i].double() for i, a in enumerate(axis)], 1)
    return torch.polar(torch.ones_like(angle), angle)[:, None]


def _exact_head(c, h, w, turn):
    if w is not None:
        h = h * (h.pow(2).mean(-1, keepdim=True) + EPS).pow(-0.5) * (w + c["offset"])
    r, p = h[..., : c["rot"]], c["rot"] // 2
    v = torch.complex(r[..., 0::2], r[..., 1::2]) if c["interleaved"] else torch.complex(r[..., :p], r[..., p:])
    v = torch.view_as_real(v * turn)
    v = v.flatten(-2) if c["interleaved"] else v.transpose(-1, -2).flatten(-2)
    return torch.cat([v, h[..., c["rot"]:]], -1)


def _exact_qk(c, s):
    D = torch.float64
    turn = _exact_turns(c, s)
    one = lambda h, w: _exact_head(c, h.to(D), None if w is None else w.to(D), turn)  # noqa: E731
    return {"q_out": one(s["q"], s["q_w"]), "k_out": one(s["k"], s["k_w"])}


def _exact_qk_bwd(c, s):
    D = torch.float64
    turn = _exact_turns(c, s)

    def one(h, w, d):
        h = h.to(D).requires_grad_(True)
        w = None if w is None else w.to(D).requires_grad_(True)
        got = torch.autograd.grad([_exact_head(c, h, w, turn)], [h] if w is None else [h, w], [d.to(D)])
        return got[0], None if w is None else got[1]

    d_q, d_q_w = one(s["q"], s["q_w"], s["d_q_out"])
    d_k, d_k_w = one(s["k"], s["k_w"], s["d_k_out"])
    return {"d_q": d_q, "d_k": d_k, "d_q_w": d_q_w, "d_k_w": d_k_w}


def _exact_layer(c, s):
    """Expert by expert over the tokens that take it."""
    D = torch.float64
    E, S, k = c["experts"], c["shared"], c["k"]
    x = s["x"].to(D)
    z = x @ s["router"].to(D).t() + s["bias"].to(D)
    top = z.topk(k, dim=1)
    share = torch.softmax(top.values, 1)
    values = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=D, device=DEV)

    def matrix(name, e):
        codes, scales = s[name + "_codes"][e].long(), s[name + "_scales"][e].view(torch.float8_e4m3fn).to(D)
        w = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=D, device=DEV)
        w[:, 0::2], w[:, 1::2] = values[codes % 16], values[codes // 16]
        return (w.view(w.shape[0], -1, 16) * scales[:, :, None]).flatten(1) * float(s[name + "_global"][e])

    out = torch.zeros_like(x) if s["residual"] is None else s["residual"].to(D)
    for e in list(range(E, E + S)) + torch.unique(top.indices).tolist():
        rows = (top.indices == e).any(1).nonzero()[:, 0] if e < E else torch.arange(c["n"], device=DEV)
        h = x[rows] @ matrix("up", e).t()
        if c["gated"]:
            g = x[rows] @ matrix("gate", e).t()
            a = g * g.sigmoid() * h
        else:
            a = h.relu().square()
        by = ((top.indices[rows] == e) * share[rows]).sum(1, keepdim=True) if e < E else 1.0
        out[rows] += by * (a @ matrix("down", e).t())
    return {"dst": out, "ids": None, "weights": share}


def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _exact_linear, "linear_bwd": _exact_linear_bwd, "qk": _exact_qk, "qk_bwd": _exact_qk_bwd,
            "layer": _exact_layer}[case["op"]](case, s)
