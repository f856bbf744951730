"""GPU: the balance loss and the router's backward pass on finite logits of any size, against the definition in 64 bits.

A row's softmax depends on differences of its logits alone.  Those of the rows here are 0, or at most 16 (multiples of
2^-4 beside an offset of 1e6, so that z - max is exact), or at least 1024 (p is 0 in 64 bits as well), so the tolerances
are those of moderate logits, as derived in test_gpu_router_loss.py."""
import pytest

from test_gpu_router_loss import Batch, _check, dev  # noqa: F401

pytestmark = pytest.mark.gpu
LOWEST = -3.4028234663852886e38  # of fp32


def _pick(b):
    """The batch's picks and weights again, from the logits that it has now."""
    import torch

    z = b.logits if b.bias is None else b.logits + b.bias
    b.ids = z.topk(b.k, dim=1).indices.to(torch.int32)
    b.weights = torch.softmax(z.gather(1, b.ids.long()), 1)
    return b


@pytest.mark.parametrize("n,E,k,ends", [(60, 40, 3, [0, 20, 60]), (33, 37, 4, None), (700, 128, 6, [0, 3, 650, 700]),
                                        (300, 256, 8, None), (200, 512, 8, [0, 77, 200]), (90, 1024, 8, None)])
@pytest.mark.parametrize("value", [-3.1e9, -1e10, -1e30, LOWEST, 5e9, 1e10, 3e38])
def test_rows_of_one_large_value(dev, n, E, k, ends, value):  # noqa: F811
    """Every expert at the same finite value, the usual way to turn all of a row off: p = 1 / E."""
    import torch

    b = Batch(dev, n, E, k, ends, 0.1, 0.0, seed=E)
    b.logits[::7] = value
    loss, counts, sums, tokens, d, db = _check(_pick(b))
    assert bool(torch.isfinite(sums).all()) and bool(torch.isfinite(d).all()) and bool(torch.isfinite(db).all())


@pytest.mark.parametrize("E", [40, 37, 128, 512])
@pytest.mark.parametrize("value", [-1e10, -1e30, LOWEST])
def test_experts_turned_off_by_a_finite_value(dev, E, value):  # noqa: F811
    """Some experts of a row, and by the bias: they have probability and gradient 0, the others share the row."""
    b = Batch(dev, 150, E, 3, [0, 50, 150], 0.1, 1.0, seed=E)
    b.logits[::2, 5:9] = value
    b.bias[11] = value
    b.bias[3] = -1.0
    b.logits[8, :] = value
    loss, counts, sums, tokens, d, db = _check(_pick(b))
    d, _ = b.backward(counts, tokens, weights=False)
    assert bool((sums[:, 11] == 0).all()) and bool((d[:8:2, 5:9] == 0).all())


@pytest.mark.parametrize("E", [40, 128, 512])
@pytest.mark.parametrize("offset", [-1e10, 1e10, -1e6, 1e6])
def test_a_common_offset(dev, E, offset):  # noqa: F811
    import torch

    b = Batch(dev, 120, E, 4, [0, 50, 120], 0.1, 0.0, seed=E)
    step = 1024.0 if abs(offset) > 1e9 else 2.0 ** -4
    few = (b.logits.clamp(-4, 4) * 16).round().clamp(-64, 64)
    b.logits = offset + few * step
    assert bool(torch.isfinite(b.logits).all())
    _check(_pick(b))


def test_the_largest_beside_the_lowest(dev):  # noqa: F811
    """z - max is below what fp32 holds."""
    b = Batch(dev, 40, 64, 3, None, 0.0, 0.0)
    b.logits[::2] = LOWEST
    b.logits[::2, 1:4] = -LOWEST
    loss, counts, sums, tokens, d, db = _check(_pick(b))
