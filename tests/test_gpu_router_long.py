"""GPU: the balance loss and the router's backward pass on batches of which a block, and a warp, has many tokens, against
the definition in 64 bits.  Tolerances as derived in test_gpu_router_loss.py: its 315 additions cover a warp's tokens (up to
6 here), 16 warps, and a join of 304 blocks in 10 additions a warp and a tree of 5."""
import pytest

from test_gpu_router_loss import Batch, _check, dev  # noqa: F401

pytestmark = pytest.mark.gpu


def _ends(n, seqs):
    """Uneven sequences, some of them empty or of one token; most boundaries inside a block's range."""
    cuts = sorted({(i * i * 7919 + 13 * i) % n for i in range(1, seqs)})
    return [0, *cuts, cuts[-1], cuts[-1] + 1, n] if cuts else [0, n]


@pytest.mark.parametrize("n", [6000, 16384, 20011])
@pytest.mark.parametrize("E,k", [(40, 3), (37, 4), (128, 8), (250, 8), (512, 8), (1024, 6)])
@pytest.mark.parametrize("seqs,masked", [(1, 0.0), (6, 0.3)])
def test_long_batches(dev, n, E, k, seqs, masked):  # noqa: F811
    _check(Batch(dev, n, E, k, _ends(n, seqs) if seqs > 1 else None, masked, 1.5, seed=n + E))


def test_many_sequences_of_a_long_batch(dev):  # noqa: F811
    """About six a block, with and without tokens."""
    n = 20000
    ends = list(range(0, n, 11))
    _check(Batch(dev, n, 96, 4, sorted(ends + ends[5::50] + [n]), 0.2, 1.0))
