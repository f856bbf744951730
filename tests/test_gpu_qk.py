"""Norms of queries and keys with rotation, forward and backward, against the definition in 64 bits.

Tolerances.  u = 2^-24 is half a step of fp32, relative.  A head's sum of squares adds at most 16 values in a lane and
four times over lanes: 21 u; the mean, eps and the inverse root 5 u more, of which the root halves all but 3: r is
within 16 u.  y = h r (offset + w) adds 4 u.  cos and sin are within 2 u of those of their argument, whose rounding to 24 bits
moves them by at most pi u (half turns up to 1, times pi), and the scale adds 1 u: 7 u of at most `scale`; the two
products and their sum 3 u.  So an output is within 32 u (|y_a| + |y_b|) scale of the definition, and rounding to bf16
adds 2^-8 of the value (2^-24 for fp32, which the 32 u hold).  Backward: dy within 10 u (|g_a| + |g_b|) scale =: of B; the
mean of w dy h r adds 21 u and 16 u and 10 u and 4 u, all of the mean of w B |h r|; r 16 u and two products: within
64 u r (w B + |h r| mean(w B |h r|)).  d_weight: a term within 32 u of B |h r|, and every addition on a value's way adds
one u: the lane's own (tokens and heads a lane takes), 32 over the block's lanes, at most 20 in each of 32 warps of the
join and 5 over those."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from nvfp4_quantized_moe_topk_gb300 import api  # noqa: E402

DEV, U, EPS = "cuda", 2.0 ** -24, 1e-6
T = {"bf16": torch.bfloat16, "fp32": torch.float32}


def rounding(t):
    return 0.0 if t == torch.float32 else torch.finfo(t).eps / 2


class Case:
    def __init__(self, n, qh, kh, D, rot, axes=1, sections=None, si=False, pi=False, dtype="bf16", norm=True, par=None,
                 offset=0.0, scale=1.0, far=4096, fused=False, seed=1):
        g = torch.Generator(device=DEV).manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
        t = T[dtype]
        self.n, self.D, self.rot, self.heads, self.dtype, self.pi = n, D, rot, (qh, kh), t, pi
        self.offset, self.scale = offset, scale
        if fused:
            rows = randn(n, (qh + 2 * kh) * D + 16).to(t)
            self.h = [rows[:, : qh * D].view(n, qh, D), rows[:, qh * D: (qh + kh) * D].view(n, kh, D)]
        else:
            self.h = [randn(n, qh, D).to(t), randn(n, kh, D).to(t)]
        self.h = [x if k else None for x, k in zip(self.h, self.heads)]
        p = T[par or dtype]
        self.w = [(randn(D) * 0.3 + 1 - offset).to(p) if norm and x is not None else None for x in self.h]
        self.g = [None if x is None else randn(*x.shape).to(t) for x in self.h]
        self.freq = (10000.0 ** (-torch.arange(rot // 2, device=DEV).double() * 2 / max(rot, 1))).float()
        self.pos = torch.randint(-far, far, (axes, n), generator=g, device=DEV, dtype=torch.int32)
        if axes == 1:
            self.pos = self.pos[0].contiguous()
        self.sections = sections
        self.kw = dict(eps=EPS, weight_offset=offset, rotary_scale=scale, sections=sections, sections_interleaved=si,
                       pairs_interleaved=pi)
        pairs = rot // 2
        if axes == 1:
            axis = [0] * pairs
        elif si:
            axis = [i % axes if i // axes < sections[i % axes] else 0 for i in range(pairs)]
        else:
            axis = [a for a, s in enumerate(sections) for _ in range(s)]
        self.angle = self.pos.view(axes, n)[axis].double().t() * self.freq.double()  # [n][pairs]

    def args(self):
        return (None, None) if not self.rot else (self.pos, self.freq)

    def forward(self):
        out = [None if x is None else torch.empty(x.shape, dtype=x.dtype, device=DEV) for x in self.h]
        api.qk_norm_rope(*self.h, *out, *self.args(), *self.w, **self.kw)
        return out

    def backward(self, **kw):
        d = [None if x is None else torch.empty(x.shape, dtype=x.dtype, device=DEV) for x in self.h]
        dw = [None if w is None else torch.empty(self.D, device=DEV) for w in self.w]
        api.qk_norm_rope_backward(*self.g, *self.h, *d, *self.args(), *self.w, *dw, **self.kw, **kw)
        return d, dw

    def split(self, x):
        r, p = x[..., : self.rot], self.rot // 2
        return (r[..., 0::2], r[..., 1::2]) if self.pi else (r[..., :p], r[..., p:])

    def merge(self, a, b, rest):
        r = torch.stack([a, b], -1).flatten(-2) if self.pi else torch.cat([a, b], -1)
        return torch.cat([r, rest], -1)

    def turned(self, x, sign=1.0):
        """x rotated, and |a| + |b| of each value's pair, in 64 bits."""
        a, b = self.split(x)
        c, s = torch.cos(self.angle)[:, None] * self.scale, sign * torch.sin(self.angle)[:, None] * self.scale
        rest = x[..., self.rot:]
        size = (a.abs() + b.abs()) * max(1.0, abs(self.scale))
        return self.merge(a * c - b * s, b * c + a * s, rest), self.merge(size, size, rest.abs())

    def reference(self, side):
        x = self.h[side].double()
        if self.w[side] is None:
            return self.turned(x)
        r = (x.pow(2).mean(-1, keepdim=True) + EPS).rsqrt()
        return self.turned(x * r * (self.w[side].double() + self.offset))

    def check(self, out=None):
        for side, got in enumerate(out or self.forward()):
            if got is None:
                continue
            ref, size = self.reference(side)
            bound = rounding(self.dtype) * ref.abs() + 32 * U * size
            assert got.dtype == self.dtype and bool(((got.double() - ref).abs() <= bound).all()), side

    def check_backward(self, got=None):
        d, dw = got or self.backward()
        for side in range(2):
            if self.h[side] is None:
                continue
            dy, B = self.turned(self.g[side].double(), -1.0)
            if self.w[side] is None:
                assert bool(((d[side].double() - dy).abs() <= rounding(self.dtype) * dy.abs() + 32 * U * B).all())
                continue
            x, w = self.h[side].double(), self.w[side].double() + self.offset
            r = (x.pow(2).mean(-1, keepdim=True) + EPS).rsqrt()
            y = x * r
            ref = r * (w * dy - y * (w * dy * y).mean(-1, keepdim=True))
            size = r * (w.abs() * B + y.abs() * (w.abs() * B * y.abs()).mean(-1, keepdim=True))
            bound = rounding(self.dtype) * ref.abs() + 64 * U * size
            assert bool(((d[side].double() - ref).abs() <= bound).all()), side
            terms, most = (dy * y).sum((0, 1)), (B * y.abs()).sum((0, 1))
            lane = -(-self.n * self.heads[side] // 8) if self.n * self.heads[side] > 4096 else 64  # (few: one warp a step)
            assert bool(((dw[side].double() - terms).abs() <= (32 + lane + 32 + 25) * U * most).all()), side


CASES = [
    dict(n=1, qh=32, kh=2, D=128, rot=128), dict(n=1, qh=1, kh=0, D=8, rot=0), dict(n=3, qh=0, kh=1, D=16, rot=16),
    dict(n=37, qh=5, kh=1, D=80, rot=80, dtype="fp32"), dict(n=37, qh=5, kh=3, D=80, rot=32, pi=True, dtype="fp32"),
    dict(n=515, qh=8, kh=2, D=64, rot=64, axes=3, sections=(8, 12, 12), offset=1.0),
    dict(n=130, qh=4, kh=4, D=128, rot=128, axes=3, sections=(24, 20, 20), si=True, fused=True),
    dict(n=61, qh=6, kh=2, D=128, rot=64, axes=2, sections=(0, 32), pi=True, scale=1.25),
    dict(n=61, qh=7, kh=2, D=256, rot=256, axes=4, sections=(32, 32, 32, 32), si=True),
    dict(n=9, qh=3, kh=1, D=72, rot=48, far=2 ** 31 - 1), dict(n=77, qh=10, kh=5, D=96, rot=96, norm=False),
    dict(n=40, qh=16, kh=8, D=192, rot=64, dtype="fp32", par="bf16", fused=True, far=2 ** 20),
    dict(n=2050, qh=12, kh=3, D=128, rot=128, par="fp32", fused=True, far=131072),
    dict(n=20, qh=9, kh=9, D=40, rot=32, norm=False, dtype="fp32", scale=0.5),
    dict(n=700, qh=3, kh=1, D=24, rot=16, pi=True), dict(n=50, qh=4, kh=2, D=248, rot=240),
]


@pytest.mark.parametrize("kw", CASES)
def test_forward(kw):
    Case(**kw).check()


@pytest.mark.parametrize("kw", CASES)
def test_backward(kw):
    Case(**kw).check_backward()


def test_gradients_against_differences():
    """The formula's gradients against central differences of the forward, both in fp32: the differences of a sum of
    products with random numbers, h = 2^-6, are off by the third derivative's h^2 (a few times 2^-12) and by the rounding of
    its terms over 2 h (2^-24 * 32 * 2^6 * a few terms of order 1)."""
    c = Case(n=2, qh=2, kh=1, D=16, rot=16, dtype="fp32", seed=7)
    d, dw = c.backward()
    value = lambda: sum(float((o.double() * g.double()).sum()) for o, g in zip(c.forward(), c.g))  # noqa: E731
    h = 2.0 ** -6
    for side in range(2):
        for x, grad in ((c.h[side], d[side]), (c.w[side], dw[side])):
            flat = x.view(-1)
            for i in range(0, flat.numel(), 5):
                old = float(flat[i])
                flat[i] = old + h
                up = value()
                flat[i] = old - h
                down = value()
                flat[i] = old
                assert abs((up - down) / (2 * h) - float(grad.view(-1)[i])) < 2e-2


def test_one_side_and_no_weights():
    c = Case(n=33, qh=4, kh=2, D=64, rot=64)
    both, (db, dwb) = c.forward(), c.backward()
    for side in range(2):
        keep = [x if i == side else None for i, x in enumerate(c.h)]
        w = [x if i == side else None for i, x in enumerate(c.w)]
        out = [None if x is None else torch.empty_like(x) for x in keep]
        api.qk_norm_rope(*keep, *out, *c.args(), *w, **c.kw)
        assert torch.equal(out[side], both[side])
        # backward: the other side's gradient missing, and each output alone
        g = [x if i == side else None for i, x in enumerate(c.g)]
        d = [torch.empty_like(x) if i == side else None for i, x in enumerate(c.h)]
        dw = [torch.empty(64, device=DEV) if i == side else None for i in range(2)]
        api.qk_norm_rope_backward(*g, *c.h, *d, *c.args(), *c.w, None, None, **c.kw)
        assert torch.equal(d[side], db[side])
        api.qk_norm_rope_backward(*g, *c.h, None, None, *c.args(), *c.w, *dw, **c.kw)
        # (other CTAs, another order of the sum)
        assert torch.allclose(dw[side], dwb[side], rtol=1e-4, atol=1e-4)


def test_in_place_and_rows_between():
    """Outputs over inputs in one projection's rows: what lies between the heads stays."""
    c = Case(n=65, qh=4, kh=2, D=64, rot=32, axes=2, sections=(7, 9), fused=True)
    want = c.forward()
    base = c.h[0]._base
    before = base.clone()
    api.qk_norm_rope(*c.h, *c.h, *c.args(), *c.w, **c.kw)
    assert torch.equal(c.h[0], want[0]) and torch.equal(c.h[1], want[1])
    assert torch.equal(base[:, 6 * 64:], before[:, 6 * 64:])
    # gradients over gradients
    c = Case(n=65, qh=4, kh=2, D=64, rot=32, axes=2, sections=(7, 9))
    d, _ = c.backward()
    dw = [torch.empty(64, device=DEV) for _ in range(2)]
    g = [x.clone() for x in c.g]
    api.qk_norm_rope_backward(*g, *c.h, *g, *c.args(), *c.w, *dw, **c.kw)
    assert torch.equal(g[0], d[0]) and torch.equal(g[1], d[1])


def test_zero_heads_infinities_and_nan():
    c = Case(n=6, qh=3, kh=1, D=64, rot=64)
    c.h[0][1, 2] = 0
    c.check()
    c.check_backward()
    clean = c.forward()
    c.h[0][2, 0, 5] = float("nan")
    c.h[0][3, 1, 7] = float("inf")
    got = c.forward()
    touched = torch.zeros(6, 3, dtype=torch.bool, device=DEV)
    touched[2, 0] = touched[3, 1] = True
    assert torch.equal(got[0][~touched], clean[0][~touched]) and torch.equal(got[1], clean[1])
    assert bool(got[0][2, 0].isnan().all()) and not bool(got[0][3, 1].isfinite().all())


def test_no_tokens():
    c = Case(n=0, qh=3, kh=1, D=64, rot=64)
    c.forward()
    d, dw = c.backward()
    assert bool((dw[0] == 0).all()) and bool((dw[1] == 0).all())


def test_same_bits_streams_and_graphs():
    c = Case(n=300, qh=8, kh=2, D=128, rot=128, axes=3, sections=(16, 24, 24))
    out, (d, dw) = c.forward(), c.backward()
    again, (d2, dw2) = c.forward(), c.backward()
    for a, b in zip([*out, *d, *dw], [*again, *d2, *dw2]):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = [torch.empty_like(x) for x in out]
    api.qk_norm_rope(*c.h, *o, *c.args(), *c.w, stream=side, **c.kw)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o[0], out[0])
    ws = api.qk_workspace(300, 8, 2, 128)
    g = torch.cuda.CUDAGraph()
    e = [torch.empty_like(x) for x in d]
    ew = [torch.empty(128, device=DEV) for _ in range(2)]
    with torch.cuda.graph(g):
        api.qk_norm_rope(*c.h, *o, *c.args(), *c.w, **c.kw)
        api.qk_norm_rope_backward(*c.g, *c.h, *e, *c.args(), *c.w, *ew, workspace=ws, **c.kw)
    for x in c.h:
        x.mul_(0.5)
    g.replay()
    want, (wd, wdw) = c.forward(), c.backward()
    for a, b in zip([*o, *e, *ew], [*want, *wd, *wdw]):
        assert torch.equal(a, b)


def test_refusals():
    c = Case(n=4, qh=3, kh=1, D=64, rot=64)
    q, k = c.h
    out = c.forward()
    ok = lambda **kw: api.qk_norm_rope(q, k, *out, *c.args(), *c.w, **{**c.kw, **kw})  # noqa: E731
    ok()
    bad = [lambda: api.qk_norm_rope(q.half(), k, *out, *c.args(), *c.w),
           lambda: api.qk_norm_rope(q, k.float(), *out, *c.args(), *c.w),
           lambda: api.qk_norm_rope(q, k, out[1], out[0], *c.args(), *c.w),
           lambda: api.qk_norm_rope(q, k, *out, c.pos, None, *c.w),
           lambda: api.qk_norm_rope(q, k, *out, c.pos.long(), c.freq, *c.w),
           lambda: api.qk_norm_rope(q, k, *out, c.pos[:3].contiguous(), c.freq, *c.w),
           lambda: api.qk_norm_rope(q, k, *out, c.pos.repeat(2, 1), c.freq, *c.w),
           lambda: api.qk_norm_rope(q, k, *out, c.pos.repeat(2, 1), c.freq, *c.w, sections=(16, 17)),
           lambda: api.qk_norm_rope(q, k, *out, c.pos.repeat(2, 1), c.freq, *c.w, sections=(32,)),
           lambda: api.qk_norm_rope(q, k, *out, c.pos, c.freq[:12], *c.w),
           lambda: api.qk_norm_rope(q.transpose(0, 1), k, *out, *c.args(), *c.w),
           lambda: api.qk_norm_rope(q, k, *out, *c.args(), c.w[0].float(), c.w[1]),
           lambda: api.qk_norm_rope(q, k, *out, *c.args(), c.w[0][:32], c.w[1]),
           lambda: ok(eps=0.0), lambda: ok(sections=(31,)),
           lambda: api.qk_norm_rope_backward(*c.g, q, k, *out, *c.args(), *c.w, torch.empty(64, device=DEV), None,
                                             workspace=torch.empty(64, dtype=torch.uint8, device=DEV)),
           lambda: api.qk_norm_rope_backward(*c.g, None, k, *out, *c.args(), *c.w)]
    for i, call in enumerate(bad):
        with pytest.raises(api.MoeError):
            call()
        torch.cuda.synchronize()
