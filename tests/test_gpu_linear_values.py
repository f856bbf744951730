"""The projections' gradients at values where their splits and activations go wrong first.  Tolerances: test_gpu_linear."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from nvfp4_quantized_moe_topk_gb300 import api  # noqa: E402
from test_gpu_linear import D, DEV, T, U, Case, half, sum_error  # noqa: E402

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
