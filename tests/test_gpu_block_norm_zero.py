"""GPU: gradients of the norms around a block through rows of zeros and of very small values, for an ordinary and a very
small eps (where such a row's 1 / rms is 1e15 and its third power more than fp32 holds), against the formulas in 64 bits;
tolerances as in test_gpu_block_norm.py."""
import pytest

from test_gpu_block_norm import Case, _check_backward, _grads, _run_backward, _run_forward, dev  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", [1e-6, 1e-30])
@pytest.mark.parametrize("H", [264, 4200])
@pytest.mark.parametrize("gate,sigmoid", [(None, False), ("channel", True), ("token", False), ("full", True)])
@pytest.mark.parametrize("small", [0.0, 2.0 ** -56])
def test_backward_of_rows_without_size(dev, eps, H, gate, sigmoid, small):  # noqa: F811
    import torch

    c = Case(dev, 40, H, "fp32", "fp32", "fp32", gate, sigmoid, beta=0.5, seed=H)
    c.kw["eps"] = eps
    c.residual[[3, 17]] *= small
    c.branch[[3, 17]] *= small
    saved = _run_forward(c)
    dr, dx = _grads(c, 4)
    got = _run_backward(c, dr, dx, saved)
    assert all(bool(torch.isfinite(v).all()) for v in got.values() if v is not None)
    _check_backward(c, dr, dx, saved, got)
