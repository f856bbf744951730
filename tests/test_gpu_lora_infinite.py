"""GPU: the adapters where the first product's result v is infinite or the largest that there is.

With positive A and B an infinite x gives an infinite v in every rank and out = y + B v is that infinity.  A finite v above
bf16's largest value (2^128 - 2^120) is v itself, not an infinity: 2^128 - 2^120 + 2^119, of 9 bits, times 2^-10 is exact
in fp32, and rounds to 2^118 in bf16 (a tie, to even)."""
import pytest

from test_gpu_lora import Case, _ids, dev  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [5, 300, 700, 5000])
@pytest.mark.parametrize("R", [16, 64, 128])
@pytest.mark.parametrize("y,o", [("bf16", "bf16"), ("fp32", "fp32"), ("fp32", "bf16")])
def test_infinite_v(dev, n, R, y, o):  # noqa: F811
    import torch

    ranks = [R, R - 3]
    c = Case(dev, [t % 2 for t in range(n)], 264, 136, 2, R, y, o, ranks, seed=R)
    c.x, c.a, c.b = (t.abs() + 0.125 for t in (c.x, c.a, c.b))
    for l in range(2):
        c.a[l, ranks[l]:] = float("nan")
        c.b[l, :, ranks[l]:] = float("nan")
    want = c.run()
    c.x[3, 7] = float("inf")
    c.x[n - 1, 201] = -float("inf")
    got = c.run()
    assert bool((got[3] == float("inf")).all()) and bool((got[n - 1] == -float("inf")).all())
    rest = torch.ones(n, dtype=torch.bool, device=dev)
    rest[[3, n - 1]] = False
    assert torch.equal(got[rest], want[rest])


@pytest.mark.parametrize("n", [5, 300, 700, 5000])
@pytest.mark.parametrize("R", [16, 64, 128])
@pytest.mark.parametrize("o", ["bf16", "fp32"])
def test_largest_v(dev, n, R, o):  # noqa: F811
    import torch

    c = Case(dev, _ids(n, 2, n, none=0.0), 264, 136, 2, R, None, o, scale=False, seed=R)
    c.x.zero_()
    c.x[:, 5] = 2.0 ** 128 - 2.0 ** 120
    c.x[:, 230] = 2.0 ** 119
    c.a.zero_()
    c.a[:, :, [5, 230]] = 1.0
    rows = torch.arange(136, device=dev)
    c.b.zero_()
    c.b[:, rows, rows % R] = 2.0 ** -10
    got = c.run()
    assert bool((got.double() == (2.0 ** 118 if o == "bf16" else 2.0 ** 118 - 2.0 ** 109)).all())
