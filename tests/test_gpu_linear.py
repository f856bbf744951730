"""Projections, forward and backward, against the definition in 64 bits.

Tolerances.  Products of bf16 are exact.  A sum of C of them runs through C / 16 instructions, each of which adds 16
products and the sum so far; what it keeps of them is open, and is taken as within 2^-22 of the largest partial sum's
bound S = sum |x w| a step, and 16 more for the parts that are joined: `sum_error`.  The activations' exponential is
within (2 + 1.2 |v|) 2^-23 of its value, its argument v for gelu within 4 * 2^-24 |v|, and a few products more: within
(8 + 6 |v|) 2^-23 of the result, and an error of z reaches it by a slope of at most 1.13 (2 |z| for relu2).  Each output is
then rounded once: 2^-8 of it for bf16.  The slope itself is within 2^-16 of 1 + |slope| for |z| < 8 (|v| < 8 wherever p (1 - p) counts: 45 units of
2^-23 in p).  A bf16 gradient is summed from dz rounded to bf16 (2^-8 of each term), an fp32 one from dz's 24 bits."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from nvfp4_quantized_moe_topk_gb300 import api  # noqa: E402

DEV, U = "cuda", 2.0 ** -24
T = {"bf16": torch.bfloat16, "fp32": torch.float32}
D = torch.float64
GELU = 2 * math.sqrt(2 / math.pi)


def half(t):
    return torch.finfo(t).eps / 2


def sum_error(C, S):
    return (C / 16 + 16) * 2.0 ** -22 * S


def act(z, name):
    if name == "relu2":
        return z.clamp(min=0).square()
    v = z if name == "silu" else GELU * (z + 0.044715 * z ** 3)
    return z if name == "none" else z * torch.sigmoid(v)


def act_error(z, dz, name):
    """How far act may be off at z, z off by dz."""
    if name == "none":
        return dz
    if name == "relu2":
        return 2 * (z.abs() + dz) * dz + 4 * U * act(z, name)
    v = z if name == "silu" else GELU * (z + 0.044715 * z ** 3)
    return 1.13 * dz + (8 + 6 * v.abs()) * 2.0 ** -23 * act(z, name).abs()


def slope(z, name):
    z = z.detach().clone().requires_grad_(True)
    return torch.autograd.grad(act(z, name).sum(), z)[0]


class Case:
    def __init__(self, n, inp, out, activation="none", bias=None, residual=None, o="bf16", z=None, scale=1.0, wide=0,
                 seed=1, dx=None, dw="bf16", in_place=False):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.randn = randn = lambda *s: torch.randn(*s, generator=g, device=DEV)
        rows = lambda r, c, t: torch.empty(r, c + wide, dtype=t, device=DEV)[:, :c]  # noqa: E731
        self.rows, self.n, self.inp, self.out_f, self.act, self.scale = rows, n, inp, out, activation, scale
        self.x, self.w = rows(n, inp, T["bf16"]), (randn(out, inp) / math.sqrt(inp)).to(T["bf16"])
        self.x.copy_(randn(n, inp))
        self.bias = None if bias is None else (randn(out) * 0.5).to(T[bias])
        self.res = None
        if residual:
            self.res = rows(n, out, T[residual])
            self.res.copy_(randn(n, out))
        self.o, self.z, self.dx, self.dw, self.in_place = T[o], z and T[z], T[dx or o], T[dw], in_place

    def forward(self):
        out = self.res if self.in_place else self.rows(self.n, self.out_f, self.o)
        z = self.rows(self.n, self.out_f, self.z) if self.z else None
        api.linear(self.x, self.w, out, self.bias, self.res, z, activation=self.act, residual_scale=self.scale)
        return out, z

    def check(self):
        x, w = self.x.to(D), self.w.to(D)
        z, err = x @ w.t(), sum_error(self.inp, x.abs() @ w.abs().t())
        if self.bias is not None:
            z, err = z + self.bias.to(D), err + U * (z.abs() + self.bias.to(D).abs())
        ref, bound = act(z, self.act), act_error(z, err, self.act)
        if self.res is not None:
            add = self.scale * self.res.to(D)
            ref, bound = ref + add, bound + 2 * U * (ref.abs() + add.abs())
        out, kept = self.forward()
        assert bool(((out.to(D) - ref).abs() <= half(self.o) * (ref.abs() + bound) + bound).all())
        if kept is not None:
            assert bool(((kept.to(D) - z).abs() <= half(self.z) * (z.abs() + err) + err).all())
        assert api.linear_device_error() == 0
        return out, kept

    def backward_inputs(self):
        self.dy = self.rows(self.n, self.out_f, self.o)
        self.dy.copy_(self.randn(self.n, self.out_f))
        self.zs = None
        if self.act != "none":
            self.zs = self.rows(self.n, self.out_f, self.z or T["bf16"])
            self.zs.copy_(self.randn(self.n, self.out_f).clamp(-7, 7))

    def backward(self, **kw):
        d_x = self.rows(self.n, self.inp, self.dx)
        d_w = torch.empty(self.out_f, self.inp, dtype=self.dw, device=DEV)
        d_b = torch.empty(self.out_f, device=DEV)
        api.linear_backward(self.dy, self.x, self.w, self.zs, d_x, d_w, d_b, activation=self.act, **kw)
        return d_x, d_w, d_b

    def check_backward(self):
        self.backward_inputs()
        d_x, d_w, d_b = self.backward()
        dz, err = self.dy.to(D), torch.zeros_like(self.dy, dtype=D)
        if self.act != "none":
            s = slope(self.zs.to(D), self.act)
            err = dz.abs() * 2.0 ** -16 * (1 + s.abs())
            dz = dz * s
        exact = self.act == "none" and self.o == torch.bfloat16
        x, w = self.x.to(D), self.w.to(D)
        for got, t, ref, size, of, C in (
                (d_x, self.dx, dz @ w, lambda e: e @ w.abs(), self.out_f, self.out_f),
                (d_w, self.dw, dz.t() @ x, lambda e: e.t() @ x.abs(), self.n, self.n)):
            terms = 1 if exact or t == torch.bfloat16 else 3
            rounded = 0.0 if exact else 2.0 ** (-8 if terms == 1 else -23)
            bound = size(err + rounded * dz.abs()) + sum_error(terms * (C + 64), size(dz.abs()))
            assert bool(((got.to(D) - ref).abs() <= half(t) * (ref.abs() + bound) + bound).all()), (t, of)
        # at most ceil(n / 64 chunks / 8 rows) + 8 + 64 additions on a value's way
        bound = err.sum(0) + (self.n / 8 + 80) * U * dz.abs().sum(0)
        assert bool(((d_b.to(D) - dz.sum(0)).abs() <= bound).all())
        assert api.linear_device_error() == 0
        return d_x, d_w, d_b


CASES = [
    dict(n=1, inp=8, out=8), dict(n=1, inp=2688, out=4608, bias="fp32"), dict(n=2, inp=64, out=128, o="fp32"),
    dict(n=7, inp=200, out=72, activation="relu2", bias="bf16", residual="bf16", scale=0.5),
    dict(n=16, inp=72, out=136, activation="silu", z="fp32", residual="fp32", o="fp32", wide=8),
    dict(n=17, inp=1000, out=520, activation="gelu_tanh", z="bf16", bias="fp32", residual="fp32", o="bf16", wide=8),
    dict(n=33, inp=1000, out=520, activation="gelu_tanh", bias="fp32", residual="fp32", o="fp32", scale=-1.5),
    dict(n=64, inp=4096, out=128, o="fp32"), dict(n=65, inp=2048, out=1032, bias="bf16", z="bf16", activation="relu2"),
    dict(n=129, inp=520, out=264, residual="bf16", in_place=True, wide=16), dict(n=200, inp=8, out=4096, o="fp32"),
    dict(n=300, inp=136, out=2000, activation="silu", bias="fp32", residual="fp32", o="fp32", in_place=True),
    dict(n=1000, inp=1032, out=1000, bias="fp32", o="fp32", wide=24),
    dict(n=2000, inp=264, out=2696, activation="gelu_tanh", z="fp32", bias="fp32"),
    dict(n=4314, inp=512, out=2688, residual="bf16"), dict(n=5000, inp=328, out=4104, activation="relu2", bias="bf16"),
]


@pytest.mark.parametrize("kw", CASES)
def test_forward(kw):
    Case(**kw).check()


BACKWARD = [
    dict(n=1, inp=8, out=8), dict(n=1, inp=264, out=72, o="fp32", dw="fp32"), dict(n=5, inp=72, out=136, dw="fp32"),
    dict(n=61, inp=1000, out=520, activation="silu", z="fp32", o="fp32", dw="fp32"),
    dict(n=64, inp=128, out=64, activation="relu2"), dict(n=65, inp=520, out=264, activation="gelu_tanh", wide=8),
    dict(n=130, inp=1000, out=200, o="fp32", dx="bf16", dw="bf16"),
    dict(n=333, inp=264, out=1032, activation="gelu_tanh", z="fp32", dx="fp32", dw="fp32", wide=8),
    dict(n=1000, inp=2000, out=1544, dw="fp32"), dict(n=2500, inp=1096, out=2056, activation="relu2", dw="fp32"),
    dict(n=4314, inp=2688, out=4608, dw="fp32"), dict(n=6000, inp=520, out=136),
]


@pytest.mark.parametrize("kw", BACKWARD)
def test_backward(kw):
    Case(**kw).check_backward()


@pytest.mark.parametrize("activation", ["none", "relu2", "silu", "gelu_tanh"])
def test_gradients_against_differences(activation):
    """Central differences of sum(out * g) over the bias's place in z, h = 2^-6: off by h^2 times the third derivative
    (below 8 on these z) and by the rounding of out over h (sums of 24 terms of order 1: 2^-23 * 64 * 24)."""
    c = Case(n=3, inp=16, out=8, activation=activation, bias="fp32", o="fp32", z="fp32")
    _, z = c.forward()
    c.dy = c.randn(3, 8)
    c.zs = None if activation == "none" else z
    d_b = c.backward()[2]
    h = 2.0 ** -6
    for i in range(8):
        value = []
        for step in (h, -2 * h):
            c.bias[i] += step
            value.append(float((c.forward()[0].to(D) * c.dy.to(D)).sum()))
        c.bias[i] += h
        assert abs((value[0] - value[1]) / (2 * h) - float(d_b[i])) < 8 * 3 * h * h * 3


def test_rows_between_and_each_output_alone():
    c = Case(n=300, inp=264, out=520, activation="silu", z="bf16", bias="fp32", wide=8)
    base = torch.full((300, 528), 7.0, dtype=torch.bfloat16, device=DEV)
    api.linear(c.x, c.w, base[:, :520], c.bias, activation="silu")
    assert bool((base[:, 520:] == 7).all())
    c.backward_inputs()
    all3 = c.backward()
    d_x, d_w, d_b = torch.empty_like(all3[0]), torch.empty_like(all3[1]), torch.empty_like(all3[2])
    api.linear_backward(c.dy, None, c.w, c.zs, d_x, activation="silu")
    api.linear_backward(c.dy, c.x, c.w, c.zs, None, d_w, activation="silu")
    api.linear_backward(c.dy, None, c.w, c.zs, None, None, d_b, activation="silu")
    assert torch.equal(d_x, all3[0]) and torch.equal(d_w, all3[1]) and torch.equal(d_b, all3[2])


def test_no_tokens():
    c = Case(n=0, inp=64, out=32)
    c.forward()
    c.dy, c.zs = torch.empty(0, 32, dtype=torch.bfloat16, device=DEV), None
    _, d_w, d_b = c.backward()
    assert bool((d_w == 0).all()) and bool((d_b == 0).all())


@pytest.mark.parametrize("n", [3, 100, 700, 4314])
def test_infinities_and_nan_stay_in_their_rows(n):
    c = Case(n=n, inp=264, out=520)
    clean = c.forward()[0].clone()
    c.x[1, 5] = float("inf")
    c.x[2, 7] = float("nan")
    got = c.forward()[0]
    assert torch.equal(got[0], clean[0]) and torch.equal(got[3:], clean[3:])
    assert not bool(got[1].isfinite().any()) and bool(got[2].isnan().all())


@pytest.mark.parametrize("n", [1, 40, 600, 4314])
def test_same_bits_streams_and_graphs(n):
    c = Case(n=n, inp=1032, out=1544, activation="gelu_tanh", z="bf16", bias="fp32", dw="fp32")
    c.backward_inputs()
    out, z = c.check()
    grads = c.backward()
    again = [*c.forward(), *c.backward()]
    for a, b in zip([out, z, *grads], again):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = torch.empty_like(out)
    api.linear(c.x, c.w, o, c.bias, activation="gelu_tanh", stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, out)
    ws = api.linear_workspace(n, 1032, 1544)
    d = [torch.empty_like(g) for g in grads]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.linear(c.x, c.w, o, c.bias, None, z, activation="gelu_tanh")
        api.linear_backward(c.dy, c.x, c.w, c.zs, *d, activation="gelu_tanh", workspace=ws)
    c.x.mul_(-0.5)
    for _ in range(2):
        graph.replay()
    want = [*c.forward(), *c.backward()]
    for a, b in zip([o, z, *d], want):
        assert torch.equal(a, b)


def test_calls_follow_one_another():
    """Products whose inputs are the outputs of the one before, back to back on one stream, large and small in turn."""
    g = torch.Generator(device=DEV).manual_seed(5)
    for n in (1, 50, 2500):
        w = [(torch.randn(o, i, generator=g, device=DEV) / math.sqrt(i)).to(torch.bfloat16)
             for i, o in ((520, 2056), (2056, 128), (128, 1032), (1032, 520))]
        x = torch.randn(n, 520, generator=g, device=DEV).to(torch.bfloat16)
        hs = [torch.empty(n, m.shape[0], dtype=torch.bfloat16, device=DEV) for m in w]
        seen = []
        for step in range(5):
            a = x
            for m, h in zip(w, hs):
                api.linear(a, m, h)
                a = h
            seen.append(a.clone())
            x = a if step % 2 else x
        torch.cuda.synchronize()  # the last step again, with the device idle between the calls
        a = seen[3]
        for m, h in zip(w, hs):
            api.linear(a, m, h)
            torch.cuda.synchronize()
            a = h.clone()
        assert torch.equal(a, seen[4])


def test_refusals():
    c = Case(n=4, inp=64, out=32)
    out = c.forward()[0]
    x, w = c.x, c.w
    bad = [lambda: api.linear(x.float(), w, out), lambda: api.linear(x, w.float(), out),
           lambda: api.linear(x, w[:, :56], out), lambda: api.linear(x, w.t(), out), lambda: api.linear(x, w, None),
           lambda: api.linear(x, w, out[:, :24]), lambda: api.linear(x, w, out.half()),
           lambda: api.linear(x, w, out, torch.zeros(31, device=DEV)),
           lambda: api.linear(x, w, out, None, out.float()[:3]), lambda: api.linear(x, w, out, z_out=out),
           lambda: api.linear(x[:, 1:].contiguous(), w, out), lambda: api.linear(x, w, out, activation="gelu"),
           lambda: api.linear(x.cpu(), w, out),
           lambda: api.linear_backward(out, x, w, None, activation="silu"),
           lambda: api.linear_backward(out, None, w, None, None, torch.empty(32, 64, device=DEV)),
           lambda: api.linear_backward(out, x, w, None, x, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))]
    for i, call in enumerate(bad):
        with pytest.raises(api.MoeError):
            call()
        torch.cuda.synchronize()


@pytest.mark.parametrize("n", [1, 15, 16, 17, 47, 48, 49, 64, 100, 128, 129])
@pytest.mark.parametrize("kw", [
    dict(inp=8, out=8, dw="fp32"), dict(inp=136, out=72, wide=8), dict(inp=264, out=200, o="fp32", dw="fp32", wide=16),
    dict(inp=1032, out=1096, activation="silu", z="fp32", dw="fp32"), dict(inp=72, out=1000, activation="relu2", dx="fp32")])
def test_gradients_of_few_tokens(n, kw):
    """Either way to d_weight: the sum of few outer products, and the larger product."""
    Case(n=n, **kw).check_backward()


@pytest.mark.parametrize("n", [5, 48, 128])
@pytest.mark.parametrize("dw", ["bf16", "fp32"])
def test_the_weight_gradient_ends_with_its_last_row(n, dw):
    c = Case(n, 136, 72, dw=dw)
    c.backward_inputs()
    room = torch.full((200, 136), 7.0, dtype=c.dw, device=DEV)
    api.linear_backward(c.dy, c.x, c.w, None, None, room[64:136], None)
    assert bool((room[:64] == 7).all()) and bool((room[136:] == 7).all())
    want = c.backward()[1]
    assert torch.equal(room[64:136], want)


@pytest.mark.parametrize("n", [3, 100])
def test_infinities_and_nan_in_few_tokens_reach_their_rows_and_columns_alone(n):
    c = Case(n, 136, 72)
    c.backward_inputs()
    clean = c.backward()[1]
    c.dy[1, 5], c.x[2, 7] = float("inf"), float("nan")
    d_w = c.backward()[1]
    touched = torch.zeros_like(clean, dtype=torch.bool)
    touched[5], touched[:, 7] = True, True
    assert not bool(torch.isfinite(d_w[5]).any()) and bool(torch.isnan(d_w[:, 7]).all())
    assert torch.equal(d_w[~touched], clean[~touched])
