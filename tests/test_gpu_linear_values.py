"""The projections' gradients at values where their splits and activations go wrong first.  Tolerances: test_gpu_linear."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from nvfp4_quantized_moe_topk_gb300 import api  # noqa: E402
from test_gpu_linear import D, DEV, GELU, T, U, Case, act, half, slope, sum_error  # noqa: E402

MOST = torch.finfo(torch.float32).max


@pytest.mark.parametrize("n", [1, 40, 100, 300])
@pytest.mark.parametrize("t", ["bf16", "fp32"])
def test_the_largest_gradients_stay_finite(n, t):
    """A d_out above the largest bf16 value, times weights and tokens of 2^-100: no term of it is infinite.  (One bf16 term of
    it is the largest bf16, within 2^-8 of it.)"""
    c = Case(n, 136, 264, o="fp32", dx=t, dw=t)
    c.backward_inputs()
    c.w[7], c.w[9], c.x[0] = 2.0 ** -100, -2.0 ** -100, 2.0 ** -100
    c.dy[0, 7], c.dy[0, 9] = MOST, -3.4e38
    d_x, d_w, d_b = c.backward()
    dz, rounded = c.dy.to(D), 2.0 ** (-8 if t == "bf16" else -23)
    for got, ref, size, C in ((d_x, dz @ c.w.to(D), lambda e: e @ c.w.to(D).abs(), 264),
                              (d_w, dz.t() @ c.x.to(D), lambda e: e.t() @ c.x.to(D).abs(), n)):
        bound = size(rounded * dz.abs()) + sum_error(3 * (C + 64), size(dz.abs()))
        assert bool(got.isfinite().all())
        assert bool(((got.to(D) - ref).abs() <= half(T[t]) * (ref.abs() + bound) + bound).all())
    assert bool(((d_b.to(D) - dz.sum(0)).abs() <= (n / 8 + 80) * U * dz.abs().sum(0)).all())


@pytest.mark.parametrize("n", [3, 100])
@pytest.mark.parametrize("t", ["bf16", "fp32"])
def test_an_infinite_gradient_stays_infinite(n, t):
    c = Case(n, 136, 72, o="fp32", dx=t, dw=t)
    c.backward_inputs()
    c.w[5], c.x[1] = c.w[5].abs() + 0.5, c.x[1].abs() + 0.5
    clean = c.backward()
    c.dy[1, 5] = float("inf")
    d_x, d_w, d_b = c.backward()
    assert bool((d_x[1] == float("inf")).all()) and bool((d_w[5] == float("inf")).all())
    rows = torch.arange(n, device=DEV) != 1
    outs = torch.arange(72, device=DEV) != 5
    assert torch.equal(d_x[rows], clean[0][rows]) and torch.equal(d_w[outs], clean[1][outs])
    assert float(d_b[5]) == float("inf") and torch.equal(d_b[outs], clean[2][outs])
    assert api.linear_device_error() == 0


@pytest.mark.parametrize("kw", [
    dict(n=512, inp=1024, out=1024, activation="silu"), dict(n=40, inp=1024, out=1024, activation="gelu_tanh", z="fp32"),
    dict(n=1000, inp=1032, out=520, activation="relu2", dw="fp32"), dict(n=700, inp=264, out=1032, o="fp32", dx="bf16")])
def test_a_bf16_gradient_is_off_by_its_own_rounding(kw):
    """The whole gradient's distance from 64 bits against that of rounding it alone.  dz in two terms adds 2^-16 of each term at
    most, 2^-17 in the mean square, against 2^-10 of the rounding: less than a thousandth; a hundredth is allowed for the sums.
    (With dz rounded to one term: 1.41 times.)"""
    c = Case(**kw)
    c.backward_inputs()
    if c.zs is not None:
        c.zs.clamp_(-3, 3)
    d_x, d_w, _ = c.backward()
    dz = c.dy.to(D)
    if c.act != "none":
        dz = dz * slope(c.zs.to(D), c.act)
    for got, ref in ((d_x, dz @ c.w.to(D)), (d_w, dz.t() @ c.x.to(D))):
        if got.dtype == torch.bfloat16:
            own = float((ref.bfloat16().to(D) - ref).norm())
            assert float((got.to(D) - ref).norm()) < 1.01 * own


@pytest.mark.parametrize("n", [64, 600])
def test_gradients_that_cancel(n):
    """Two features with the same weights and opposite gradients, but for 2^-12 of them: what is left is right to 2^-2 where dz
    holds 2^-16 of each term, and nothing is where it holds 2^-8."""
    c = Case(n, 264, 136, o="fp32", dx="bf16", dw="bf16")
    c.backward_inputs()
    c.w[1::2] = c.w[0::2]
    c.dy[:, 1::2] = -c.dy[:, 0::2] * (1 + 2.0 ** -12)
    d_x = c.backward()[0]
    dz, w = c.dy.to(D), c.w.to(D)
    ref, size = dz @ w, dz.abs() @ w.abs()
    bound = 2.0 ** -16 * size + sum_error(2 * (136 + 64), size)
    assert bool(((d_x.to(D) - ref).abs() <= 2.0 ** -8 * (ref.abs() + bound) + bound).all())
    assert float((d_x.to(D) - ref).norm()) < 2.0 ** -2 * float(ref.norm())


def _long(n, inp, out, o):
    """All values positive, rows of many sizes: a sum that is cut on the way shows in full."""
    g = torch.Generator(device=DEV).manual_seed(7)
    x = (torch.rand(n, inp, generator=g, device=DEV) + 0.5) * (1 + torch.rand(n, 1, generator=g, device=DEV))
    w = torch.rand(out, inp, generator=g, device=DEV) + 0.5
    return x.bfloat16(), w.bfloat16(), torch.empty(n, out, dtype=T[o], device=DEV)


def _exact(x, w):
    ref = torch.zeros(x.shape[0], w.shape[0], dtype=D, device=DEV)
    for c in range(0, x.shape[1], 1 << 16):
        ref += x[:, c: c + (1 << 16)].to(D) @ w[:, c: c + (1 << 16)].to(D).t()
    return ref


@pytest.mark.parametrize("n,inp,out,o", [(200, 1 << 20, 8, "bf16"), (200, 1 << 20, 264, "bf16"), (40, (1 << 20) + 72, 4096, "bf16"),
                                         (4, 1 << 22, 8, "fp32"), (4, 1 << 22, 8, "bf16"), (33, 1 << 21, 24, "fp32")])
def test_long_sums(n, inp, out, o):
    """Short chains, each within 36 steps of 2^-22 of itself, whose sums are added in fp32, a rounding of 2^-24 each: C / 512 of
    them, in the way of up to 16 tokens and 64 features an eighth as many in each of 8 warps.  (A sum cut all the way is 1e-9 a
    column off.)"""
    x, w, out_t = _long(n, inp, out, o)
    api.linear(x, w, out_t)
    ref = _exact(x, w)
    own = 36 * 2.0 ** -22 + (inp / 512 / (8 if out <= 64 and n <= 64 else 1) + 16) * U
    assert bool(((out_t.to(D) - ref).abs() <= (half(T[o]) + own) * (1 + 2.0 ** -7) * ref).all())
    assert api.linear_device_error() == 0


@pytest.mark.parametrize("dw", ["bf16", "fp32"])
def test_long_sums_of_tokens(dw):
    n = (1 << 20) + 24
    x, w, _ = _long(16, n, 72, "bf16")
    x, dy = x.t().contiguous(), w.t().contiguous()  # d_weight [72, 16] of n tokens
    d_w = torch.empty(72, 16, dtype=T[dw], device=DEV)
    api.linear_backward(dy, x, torch.zeros(72, 16, dtype=torch.bfloat16, device=DEV), None, None, d_w)
    ref = _exact(dy.t(), x.t())
    own = 36 * 2.0 ** -22 + (n / 512 + 16) * U
    assert bool(((d_w.to(D) - ref).abs() <= (half(T[dw]) + own) * (1 + 2.0 ** -7) * ref).all())


@pytest.mark.parametrize("activation", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("n", [1, 40, 100, 2500])
def test_activations_far_below_zero(n, activation):
    """Where exp(-v) overflows or nears it, the value is still a number that fp32 holds.  To test_gpu_linear's (8 + 6 |v|) 2^-23
    an exponential below the smallest normal number adds 2^-149 of its factor."""
    out = 2056
    lo, hi = (-104.0, -60.0) if activation == "silu" else (-10.6, -8.8)
    z = torch.linspace(lo, hi, out, device=DEV)
    x, w = torch.zeros(n, 8, dtype=torch.bfloat16, device=DEV), torch.zeros(out, 8, dtype=torch.bfloat16, device=DEV)
    got, kept = torch.empty(n, out, device=DEV), torch.empty(n, out, device=DEV)
    api.linear(x, w, got, z, None, kept, activation=activation)
    assert torch.equal(kept, z.expand(n, out))
    zd = z.to(D)
    v = (zd if activation == "silu" else GELU * (zd + 0.044715 * zd ** 3)).abs()
    ref = act(zd, activation)
    assert bool(((got.to(D) - ref).abs() <= (8 + 6 * v) * 2.0 ** -23 * ref.abs() + 2.0 ** -148 * (1 + zd.abs())).all())
    assert bool((got[:, ref.abs() > 2.0 ** -126] != 0).all())
    dy, d_b = torch.ones(n, out, device=DEV), torch.empty(out, device=DEV)
    api.linear_backward(dy, None, w, kept, None, None, d_b, activation=activation)
    s = slope(zd, activation)
    size = v if activation == "silu" else GELU * zd.abs() * (1 + 3 * 0.044715 * zd ** 2)  # of p and of z p
    bound = (8 + 6 * v + n / 8 + 80) * 2.0 ** -23 * s.abs() + 2.0 ** -148 * (1 + size)
    assert bool(((d_b.to(D) - n * s).abs() <= n * bound).all())
    assert bool((d_b[s.abs() > 2.0 ** -126] != 0).all())


@pytest.mark.parametrize("n", [1 << 12, (1 << 20) + 5, 1 << 24])
def test_column_sums_of_many_tokens(n):
    """d_bias of equal gradients, which round the same way at every addition once their sum has few bits left for them.  A thread
    adds 64 rows, such sums of its n / 2432 rows, then 8 threads', 304 chunks' by 32 warps and those: a rounding of 2^-24 each."""
    dy = torch.full((n, 8), 1 + 0.98 * 2.0 ** -12, device=DEV)
    dy[:, 4:] *= -3
    w, d_b = torch.zeros(8, 8, dtype=torch.bfloat16, device=DEV), torch.empty(8, device=DEV)
    api.linear_backward(dy, None, w, None, None, None, d_b)
    ref = dy[0].to(D) * n
    assert bool(((d_b.to(D) - ref).abs() <= (64 + n / 2432 / 64 + 1 + 8 + 10 + 5) * U * ref.abs()).all())


@pytest.mark.parametrize("n", [3, 100])
@pytest.mark.parametrize("value", [float("nan"), float("-inf")])
@pytest.mark.parametrize("dx,dw", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "bf16")])
def test_a_gradient_that_is_no_number_stays_in_its_row(n, value, dx, dw):
    c = Case(n, 136, 72, activation="relu2", z="fp32", o="fp32", dx=dx, dw=dw)
    c.backward_inputs()
    c.w[5], c.x[1], c.zs[1, 5] = c.w[5].abs() + 0.5, c.x[1].abs() + 0.5, 1.0
    clean = c.backward()
    c.dy[1, 5] = value
    d_x, d_w, d_b = c.backward()
    rows, outs = torch.arange(n, device=DEV) != 1, torch.arange(72, device=DEV) != 5
    assert torch.equal(d_x[rows], clean[0][rows]) and torch.equal(d_w[outs], clean[1][outs])
    for got in (d_x[1], d_w[5], d_b[5]):
        assert bool((got.isnan() if value != value else got == value).all())


@pytest.mark.parametrize("kw", [
    dict(n=100, inp=(1 << 19) + 8, out=136, activation="relu2", z="bf16", bias="fp32", residual="bf16"),
    dict(n=70, inp=1 << 19, out=72, activation="silu", bias="bf16", residual="fp32", scale=0.5, wide=8),
    dict(n=9, inp=40000, out=520, activation="gelu_tanh", z="fp32", residual="bf16", o="fp32")])
def test_epilogues_behind_long_sums(kw):
    Case(**kw).check()


@pytest.mark.parametrize("n", [20, 100, 700])
def test_gradients_of_two_types_are_those_of_each_alone(n):
    """dz in three terms for one gradient: the other takes the first two, the same as by itself."""
    c = Case(n, 264, 520, activation="silu", dx="bf16", dw="fp32")
    c.backward_inputs()
    d_x, d_w, d_b = c.backward()
    x, w, b = torch.empty_like(d_x), torch.empty_like(d_w), torch.empty_like(d_b)
    api.linear_backward(c.dy, None, c.w, c.zs, x, activation="silu")
    api.linear_backward(c.dy, c.x, c.w, c.zs, None, w, activation="silu")
    api.linear_backward(c.dy, None, c.w, c.zs, None, None, b, activation="silu")
    assert torch.equal(x, d_x) and torch.equal(w, d_w) and torch.equal(b, d_b)
