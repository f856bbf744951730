"""GPU parity of the norms around a block (moe_block_norm, moe_block_norm_backward) with the formulas in 64 bits.

Tolerances.  The kernels work in fp32 and round each output once.  Every output is a short chain of fp32 operations on
terms whose absolute values a reference can add up (``scale`` below: the formula with every term's absolute value); a
chain of k operations moves the result by at most k 2^-24 of that.  The longest chain has about 20 links plus half of
the relative error of a mean of H squares summed in runs of at most 16 and a tree (under 32 links): 64 2^-24 = 4e-6.
bf16 outputs add half a unit in the last place, at most 2^-8 of the value."""
import pytest

pytestmark = pytest.mark.gpu
EPS = 1e-6
CHAIN = 4e-6


@pytest.fixture(scope="module")
def dev():
    import torch

    from nvfp4_quantized_moe_topk_gb300 import api

    api.load(build_if_missing=True)
    return torch.device("cuda:0")


def _types(name):
    import torch

    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


class Case:
    """Inputs of one call, and the reference's values and scales in 64 bits."""

    def __init__(self, dev, n, H, res="bf16", act="bf16", par="bf16", gate=None, sigmoid=False, post=True, pre=True,
                 branch=True, alpha=1.0, beta=1.0, offset=0.0, seed=0):
        import torch

        g = torch.Generator(device=dev).manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
        self.n, self.H, self.sigmoid, self.alpha, self.beta, self.offset = n, H, sigmoid, alpha, beta, offset
        self.res, self.act, self.par = _types(res), _types(act), _types(par)
        self.residual = (2 * r(n, H)).to(self.res)
        self.branch = r(n, H).to(self.act) if branch else None
        self.post = (1 - offset + 0.2 * r(H)).to(self.par) if post and branch else None
        self.pre = (1 - offset + 0.2 * r(H)).to(self.par) if pre else None
        shape = {None: None, "channel": (H,), "token": (n, 1), "full": (n, H)}[gate if branch else None]
        kind = {"channel": self.par, "token": torch.float32, "full": self.act}.get(gate)
        self.gate = None if shape is None else r(*shape).to(kind)
        self.kw = dict(eps=EPS, residual_scale=alpha, branch_scale=beta, weight_offset=offset, gate_sigmoid=sigmoid)

    def g64(self):
        if self.gate is None:
            return 1.0
        g = self.gate.double()
        return g.sigmoid() if self.sigmoid else g

    def forward64(self, residual=None, branch=None, post=None, pre=None, gate=None):
        """(u, x, rp, ru, scale of u); x, rp, ru None where there are none."""
        residual = self.residual.double() if residual is None else residual
        branch = self.branch.double() if branch is None and self.branch is not None else branch
        post = self.post.double() if post is None and self.post is not None else post
        pre = self.pre.double() if pre is None and self.pre is not None else pre
        gate = self.g64() if gate is None else gate
        rp = ru = x = None
        u = self.alpha * residual
        scale = u.abs()
        if branch is not None:
            z = branch
            if post is not None:
                rp = (branch.square().mean(1, keepdim=True) + EPS).rsqrt()
                z = z * rp * (post + self.offset)
            z = self.beta * gate * z
            u = u + z
            scale = scale + z.abs()
        if pre is not None:
            ru = (u.square().mean(1, keepdim=True) + EPS).rsqrt()
            x = u * ru * (pre + self.offset)
        return u, x, rp, ru, scale


def _close(got, want, scale, where, chain=CHAIN):
    import torch

    assert got.shape == want.shape, where
    tol = chain * scale + 1e-30
    if got.dtype == torch.bfloat16:
        tol = tol + want.abs() * 2.0 ** -8
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), (where, float((err / tol).max()), float(err.max()))


def _run_forward(c, out=None, x=None, stream=None):
    import torch

    from nvfp4_quantized_moe_topk_gb300 import api

    dev = c.residual.device
    out = torch.full((c.n, c.H), 7.0, dtype=c.res, device=dev) if out is None else out
    x = (torch.full((c.n, c.H), 7.0, dtype=torch.bfloat16, device=dev) if x is None else x) if c.pre is not None else None
    rp = torch.empty(c.n, device=dev) if c.post is not None else None
    ru = torch.empty(c.n, device=dev) if c.pre is not None else None
    got = api.block_norm(c.residual, c.branch, c.gate, c.post, c.pre, out, x, rp, ru, stream=stream, **c.kw)
    assert got[0] is out and got[1] is x
    return out, x, rp, ru


def _check_forward(c, out, x, rp, ru):
    u, xr, rpr, rur, scale = c.forward64()
    _close(out, u, scale, "residual_out")
    if rpr is not None:
        _close(rp, rpr[:, 0], rpr[:, 0], "rstd_post")
    if xr is not None:
        _close(ru, rur[:, 0], rur[:, 0] * (1 + (scale.square().sum(1) / u.square().sum(1).clamp(min=1e-30)).sqrt()),
               "rstd_pre")
        w = (c.pre.double() + c.offset).abs()
        worst = (scale.square().mean(1, keepdim=True) + EPS).sqrt() * rur
        _close(x, xr, (scale + u.abs() * worst) * rur * w + xr.abs(), "x_out")


SIZES = [(1, 8), (2, 64), (33, 256), (5, 1000), (3, 2688), (61, 4096), (2, 4104), (3, 8192), (700, 264)]


@pytest.mark.parametrize("n,H", SIZES)
@pytest.mark.parametrize("res,act", [("bf16", "bf16"), ("fp32", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
def test_forward_sizes_and_types(dev, n, H, res, act):
    c = Case(dev, n, H, res, act, par="fp32" if n % 2 else "bf16", gate="channel", beta=0.5, seed=n + H)
    _check_forward(c, *_run_forward(c))


@pytest.mark.parametrize("gate", [None, "channel", "token", "full"])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("H", [1000, 4200])
def test_forward_gates(dev, gate, sigmoid, post, H):
    c = Case(dev, 9, H, "fp32", "bf16", "bf16", gate, sigmoid and gate is not None, post, alpha=1.5, beta=-0.25,
             offset=1.0, seed=3)
    _check_forward(c, *_run_forward(c))


def test_forward_before_a_block_alone(dev):
    """No branch: the pre-norm (with the residual scale), residual_out optional."""
    import torch

    from nvfp4_quantized_moe_topk_gb300 import api

    c = Case(dev, 17, 2688, branch=False, alpha=0.5)
    _check_forward(c, *_run_forward(c))
    x = torch.empty(17, 2688, dtype=torch.bfloat16, device=dev)
    api.block_norm(c.residual, pre_weight=c.pre, x_out=x, **c.kw)
    assert torch.equal(x, _run_forward(c)[1])


def test_forward_after_a_block_alone_in_place(dev):
    """No pre-norm; residual_out is residual."""
    import torch

    c = Case(dev, 40, 2688, "fp32", "bf16", gate="token", sigmoid=True, pre=False)
    want = _run_forward(c)[0].clone()
    u, _, _, _, scale = c.forward64()
    _close(want, u, scale, "residual_out")
    _run_forward(c, out=c.residual)
    assert torch.equal(c.residual, want)


def test_forward_row_strides(dev):
    """Every matrix is a slice of a wider one; what lies beside the slices is left alone."""
    import torch

    c = Case(dev, 21, 264, gate="full")
    plain = _run_forward(c)
    wide = torch.full((21, 5, 280), 3.0, dtype=torch.bfloat16, device=dev)
    views = [wide[:, i, 8:272] for i in range(5)]
    for v, t in zip(views, (c.residual, c.branch, c.gate)):
        v.copy_(t)
    c.residual, c.branch, c.gate = views[:3]
    got = _run_forward(c, out=views[3], x=views[4])
    assert all(torch.equal(a, b) for a, b in zip(plain, got))
    assert bool((wide[:, :, :8] == 3).all()) and bool((wide[:, :, 272:] == 3).all())


def test_zero_rows_and_bad_rows_stay_to_themselves(dev):
    """A row of zeros gives zeros; an infinite or NaN row does not reach its neighbours."""
    import torch

    c = Case(dev, 6, 2688, "fp32", "fp32", "fp32")
    clean = _run_forward(c)
    c.residual[1] = 0
    c.branch[1] = 0
    c.residual[3, 5] = float("nan")
    c.branch[4, 7] = float("inf")
    got = _run_forward(c)
    assert bool((got[0][1] == 0).all()) and bool((got[1][1] == 0).all())
    assert abs(float(got[3][1]) - EPS ** -0.5) < 1e-4 * EPS ** -0.5
    assert bool(torch.isnan(got[1][3]).all()) and bool(torch.isnan(got[1][4].float()).any())
    for i in (0, 2, 5):
        assert torch.equal(got[0][i], clean[0][i]) and torch.equal(got[1][i], clean[1][i])


def test_offsets_past_32_bits(dev):
    """2.2e9 elements a matrix: the last rows against the formula."""
    import torch

    from nvfp4_quantized_moe_topk_gb300 import api

    n, H = 270000, 8192
    assert n * H > 2 ** 31
    r = torch.zeros(n, H, dtype=torch.bfloat16, device=dev)
    small = Case(dev, 3, H, branch=False)
    r[-3:] = small.residual
    x = torch.empty_like(r)
    ru = torch.empty(n, device=dev)
    api.block_norm(r, pre_weight=small.pre, x_out=x, rstd_pre=ru, eps=EPS)
    want = _run_forward(small)
    assert torch.equal(x[-3:], want[1]) and torch.equal(ru[-3:], want[3])
    assert bool((x[:-3:5000] == 0).all())


# ------------------------------------------------------------------ backward

def _run_backward(c, dr, dx, saved, stream=None, workspace=None, inplace=False):
    import torch

    from nvfp4_quantized_moe_topk_gb300 import api

    dev = c.residual.device
    out, _, rp, ru = saved
    d_res = dr if inplace else torch.full((c.n, c.H), 7.0, dtype=c.res, device=dev)
    d_br = (c.branch if inplace else torch.full((c.n, c.H), 7.0, dtype=c.act, device=dev)) \
        if c.branch is not None else None
    d_gate = None
    if c.gate is not None:
        d_gate = torch.full(c.gate.shape, 7.0, dtype=c.act if c.gate.shape == (c.n, c.H) else torch.float32, device=dev)
    d_post = torch.full((c.H,), 7.0, device=dev) if c.post is not None else None
    d_pre = torch.full((c.H,), 7.0, device=dev) if c.pre is not None and dx is not None else None
    api.block_norm_backward(dr, dx, out, c.branch, c.gate, c.post, c.pre if dx is not None else None, rp, ru, d_res,
                            d_br, d_gate, d_post, d_pre, stream=stream, workspace=workspace, **c.kw)
    return dict(d_residual=d_res, d_branch=d_br, d_gate=d_gate, d_post=d_post, d_pre=d_pre)


def _reference_backward(c, dr, dx, saved):
    """{name: (value, scale)} by the formulas on what the forward saved."""
    import torch

    out, _, rp, ru = saved
    zero = torch.zeros(c.n, c.H, dtype=torch.float64, device=c.residual.device)
    G = zero if dr is None else dr.double()
    S = G.abs()
    r = {}
    if dx is not None:
        h, w, d = out.double() * ru.double()[:, None], c.pre.double() + c.offset, dx.double()
        q = w * d
        G = G + ru.double()[:, None] * (q - h * (q * h).mean(1, keepdim=True))
        S = S + ru.double()[:, None] * (q.abs() + h.abs() * (q * h).abs().mean(1, keepdim=True))
        r["d_pre"] = ((d * h).sum(0), (d * h).abs().sum(0))
    r["d_residual"] = (c.alpha * G, abs(c.alpha) * S)
    if c.branch is None:
        return r
    yh = c.branch.double() * (1.0 if c.post is None else rp.double()[:, None])
    w = torch.ones(c.H, dtype=torch.float64, device=yh.device) if c.post is None else c.post.double() + c.offset
    g = c.g64() * torch.ones_like(yh)
    dz, Sz = c.beta * g * G, abs(c.beta) * g.abs() * S
    if c.post is None:
        r["d_branch"] = (dz, Sz)
    else:
        m, Sm = (w * dz * yh).mean(1, keepdim=True), (w * yh).abs().mul(Sz).mean(1, keepdim=True)
        rp1 = rp.double()[:, None]
        r["d_branch"] = (rp1 * (w * dz - yh * m), rp1 * (w.abs() * Sz + yh.abs() * Sm))
        r["d_post"] = ((dz * yh).sum(0), (Sz * yh.abs()).sum(0))
    if c.gate is not None:
        f = g * (1 - g) if c.sigmoid else torch.ones_like(g)
        dg, Sg = c.beta * yh * w * G * f, abs(c.beta) * (yh * w * f).abs() * S
        if c.gate.dim() == 1:
            dg, Sg = dg.sum(0), Sg.sum(0)
        elif c.gate.shape == (c.n, 1):
            dg, Sg = dg.sum(1, keepdim=True), Sg.sum(1, keepdim=True)
        r["d_gate"] = (dg, Sg)
    return r


def _check_backward(c, dr, dx, saved, got):
    for name, (want, scale) in _reference_backward(c, dr, dx, saved).items():
        # two chains follow one another (G, then what is made of it); sums over tokens add at most 3 (rows of a CTA,
        # here up to 3) + 19 (CTAs of a warp) + 16 (warps) links
        _close(got[name], want, scale, name, chain=3 * CHAIN)


def _grads(c, seed, dx=True):
    import torch

    g = torch.Generator(device=c.residual.device).manual_seed(seed)
    dr = torch.randn(c.n, c.H, generator=g, device=c.residual.device).to(c.res)
    return dr, torch.randn(c.n, c.H, generator=g, device=c.residual.device).to(torch.bfloat16) if dx else None


@pytest.mark.parametrize("n,H", SIZES)
@pytest.mark.parametrize("res,act", [("bf16", "bf16"), ("fp32", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
def test_backward_sizes_and_types(dev, n, H, res, act):
    c = Case(dev, n, H, res, act, par="fp32" if n % 2 else "bf16", gate="channel", beta=0.5, seed=n + H)
    saved = _run_forward(c)
    dr, dx = _grads(c, 5)
    _check_backward(c, dr, dx, saved, _run_backward(c, dr, dx, saved))


@pytest.mark.parametrize("gate", [None, "channel", "token", "full"])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("H", [1000, 4200])
def test_backward_gates(dev, gate, sigmoid, post, H):
    c = Case(dev, 9, H, "fp32", "bf16", "bf16", gate, sigmoid and gate is not None, post, alpha=1.5, beta=-0.25,
             offset=1.0, seed=3)
    saved = _run_forward(c)
    dr, dx = _grads(c, 6)
    _check_backward(c, dr, dx, saved, _run_backward(c, dr, dx, saved))


def test_backward_of_each_side_alone(dev):
    import torch

    # after a block alone: no x, no gradient through the second norm
    c = Case(dev, 40, 2688, gate="token", sigmoid=True, pre=False)
    saved = _run_forward(c)
    dr, _ = _grads(c, 7, dx=False)
    _check_backward(c, dr, None, saved, _run_backward(c, dr, None, saved))
    # before a block alone, no gradient of residual_out
    c = Case(dev, 40, 2688, branch=False)
    saved = _run_forward(c)
    _, dx = _grads(c, 8)
    got = _run_backward(c, None, dx, saved)
    _check_backward(c, None, dx, saved, got)
    assert got["d_branch"] is None and bool(torch.isfinite(got["d_residual"]).all())


def test_backward_in_place_and_repeated(dev):
    import torch

    from nvfp4_quantized_moe_topk_gb300 import api

    c = Case(dev, 650, 2688, gate="channel")
    saved = _run_forward(c)
    dr, dx = _grads(c, 9)
    ws = api.block_norm_workspace(c.n, c.H)
    want = _run_backward(c, dr, dx, saved, workspace=ws)
    ws.fill_(0xFF)
    again = _run_backward(c, dr, dx, saved, workspace=ws)
    assert all(torch.equal(want[k], again[k]) for k in want)
    place = _run_backward(c, dr, dx, saved, inplace=True)
    assert all(torch.equal(want[k], place[k]) for k in want)


def test_backward_of_no_tokens_zeroes_the_sums(dev):
    c = Case(dev, 0, 264, gate="channel")
    dr, dx = _grads(c, 1)
    got = _run_backward(c, dr, dx, _run_forward(c))
    for k in ("d_gate", "d_post", "d_pre"):
        assert bool((got[k] == 0).all()), k


@pytest.mark.parametrize("gate,sigmoid", [("channel", True), ("token", False), ("full", True)])
def test_backward_against_differences(dev, gate, sigmoid):
    """<gradient, direction> against a central difference of L = sum(u dr) + sum(x dx) in 64 bits, one input at a time.
    All stored values are fp32, so the saved row statistics are within 1e-6 of the formula's; the difference's own error
    is h^2 ~ 1e-8 relative: 1e-4 of the sum of the terms' absolute values is ample for both."""
    import torch

    c = Case(dev, 7, 264, "fp32", "fp32", "fp32", gate, sigmoid, alpha=1.25, beta=0.5)
    saved = _run_forward(c)
    dr, dx = _grads(c, 11)
    got = _run_backward(c, dr, dx, saved)
    g = torch.Generator(device=dev).manual_seed(12)
    leaves = dict(residual=c.residual, branch=c.branch, post=c.post, pre=c.pre, gate=c.gate)
    names = dict(residual="d_residual", branch="d_branch", post="d_post", pre="d_pre", gate="d_gate")
    for name, t in leaves.items():
        v = torch.randn(t.shape, generator=g, device=dev, dtype=torch.float64)

        def L(h):
            p = t.double() + h * v
            if name == "gate" and sigmoid:
                p = p.sigmoid()
            u, x, _, _, _ = c.forward64(**{name: p})
            return (u * dr.double()).sum() + (x * dx.double()).sum()

        h = 1e-4
        diff = float((L(h) - L(-h)) / (2 * h))
        terms = got[names[name]].double() * v
        assert abs(float(terms.sum()) - diff) <= 1e-4 * float(terms.abs().sum()), name


def test_on_another_stream(dev):
    """Everything on a stream that is not the current one, the workspace allocated by the call."""
    import torch

    c = Case(dev, 300, 2688, gate="channel")
    saved = _run_forward(c)
    dr, dx = _grads(c, 13)
    want = _run_backward(c, dr, dx, saved)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for handle in (s, s.cuda_stream):
        with torch.cuda.stream(s):  # the buffers that the helpers fill belong to s as well
            fw = _run_forward(c, stream=handle)
            got = _run_backward(c, dr, dx, saved, stream=handle)
        s.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(fw, saved))
        assert all(torch.equal(want[k], got[k]) for k in want)
    out = [torch.empty_like(t) for t in saved]
    torch.cuda.synchronize()
    from nvfp4_quantized_moe_topk_gb300 import api

    api.block_norm(c.residual, c.branch, c.gate, c.post, c.pre, *out, stream=s, **c.kw)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(out, saved))


def test_refusals(dev):
    import torch

    from nvfp4_quantized_moe_topk_gb300 import api

    c = Case(dev, 4, 264, gate="channel")
    ok = dict(residual=c.residual, branch=c.branch, gate=c.gate, post_weight=c.post, pre_weight=c.pre,
              residual_out=torch.empty_like(c.residual), x_out=torch.empty_like(c.residual))
    api.block_norm(**ok)
    bad = [dict(residual=c.residual.half()), dict(residual=c.residual.cpu()), dict(branch=c.branch[:3]),
           dict(branch=c.branch.float().double()), dict(gate=c.gate[:8]), dict(post_weight=c.post.float()),
           dict(x_out=torch.empty(4, 264, device=dev)), dict(x_out=None), dict(eps=0.0), dict(eps=float("nan")),
           dict(residual_out=c.residual[:1].expand(4, 264)), dict(residual=c.residual.t().contiguous().t()),
           dict(branch=None), dict(rstd_pre=torch.empty(5, device=dev)), dict(pre_weight=None)]
    for b in bad:
        with pytest.raises(api.MoeError):
            api.block_norm(**dict(ok, **b))
    for H in (12, 8200):
        with pytest.raises(api.MoeError) as e:
            t = torch.zeros(2, H, dtype=torch.bfloat16, device=dev)
            api.block_norm(t, pre_weight=t[0], x_out=torch.empty_like(t))
        assert e.value.status == 2
    # a misaligned row start
    flat = torch.zeros(4 * 264 + 8, dtype=torch.bfloat16, device=dev)
    with pytest.raises(api.MoeError):
        api.block_norm(**dict(ok, residual=flat[1:1 + 4 * 264].view(4, 264)))
    saved = _run_forward(c)
    dr, dx = _grads(c, 1)
    with pytest.raises(api.MoeError) as e:
        _run_backward(c, dr, dx, saved, workspace=torch.empty(64, dtype=torch.uint8, device=dev))
    assert e.value.status == 3
    with pytest.raises(api.MoeError):
        _run_backward(c, dr, dx, (saved[0], None, None, saved[3]))
    with pytest.raises(api.MoeError):
        api.block_norm_backward(dr, dx, saved[0], c.branch, c.gate, c.post, c.pre, saved[2], saved[3],
                                d_gate=torch.empty(4, 1, device=dev))
