"""GPU: the norms around a block where a CTA works on several rows, against the formulas in 64 bits.

Sizes: with 152 SMs the forward pass runs at most 1216 CTAs at 1000 channels, 304 at 2688 and 152 at 4200 and 8192, the
backward pass at most 912, 304, 152 and 152: the batches here have three to sixteen rows for each.  Rows do not depend on
one another, so the tolerances are those of test_gpu_block_norm.py; column sums add up to 17 rows of a CTA, 10 CTAs of a
warp and a tree of 5, inside its 3 x 64 links."""
import pytest

from test_gpu_block_norm import Case, _check_backward, _check_forward, _grads, _run_backward, _run_forward, dev  # noqa: F401

pytestmark = pytest.mark.gpu


def _both(c, seed=5, dx=True):
    saved = _run_forward(c)
    _check_forward(c, *saved)
    dr, dx = _grads(c, seed, dx)
    _check_backward(c, dr, dx, saved, _run_backward(c, dr, dx, saved))


@pytest.mark.parametrize("n,H", [(5000, 1000), (2500, 2688), (2500, 4200)])
@pytest.mark.parametrize("gate,sigmoid", [(None, False), ("channel", False), ("channel", True), ("token", False),
                                          ("token", True), ("full", False), ("full", True)])
@pytest.mark.parametrize("res,act", [("bf16", "bf16"), ("fp32", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
def test_gates(dev, n, H, gate, sigmoid, res, act):  # noqa: F811
    _both(Case(dev, n, H, res, act, "fp32", gate, sigmoid, alpha=1.5, beta=-0.5, seed=H))


@pytest.mark.parametrize("n,H", [(5000, 1000), (2500, 2688), (2500, 4200)])
@pytest.mark.parametrize("gate", [None, "token", "full"])
def test_one_norm_alone(dev, n, H, gate):  # noqa: F811
    _both(Case(dev, n, H, "fp32", "bf16", gate=gate, pre=False, seed=1), dx=False)
    _both(Case(dev, n, H, gate=gate, post=False, seed=2))
    _both(Case(dev, n, H, "fp32", branch=False, seed=3))


def test_one_ring_stage(dev):  # noqa: F811
    """fp32 rows of 8192 channels with a full gate: the backward pass has room for a single stage."""
    _both(Case(dev, 700, 8192, "fp32", "fp32", "fp32", "full", True))


def test_narrow_rows(dev):  # noqa: F811
    _both(Case(dev, 9000, 264, gate="channel", beta=0.5))
