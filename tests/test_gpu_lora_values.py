"""GPU: what the adapters' first product hands to the second (v) keeps all its bits.

Here every token's x has three entries, k0 2^14, k1 2^7 and k2 with 1 <= k < 128, at columns where A is 1 or -1: every
product, partial sum and v is an integer below 2^21, B and the scales are powers of two with one entry of B a row, and y
takes v's leading part away.  fp32 holds each step exactly in whatever order it is done, so the result is the definition's,
rounded once: equal, without a tolerance."""
import pytest

from test_gpu_lora import Case, _ids, dev  # noqa: F401

pytestmark = pytest.mark.gpu

SIZES = [(1, 2, 16, 72, 40), (40, 3, 32, 1000, 136), (40, 5, 128, 264, 72), (300, 4, 16, 264, 136), (700, 3, 64, 520, 136),
         (700, 3, 128, 520, 264), (2100, 2, 8, 136, 72), (5000, 3, 64, 264, 136), (5000, 3, 128, 264, 136),
         (12400, 4, 128, 328, 136), (12400, 4, 32, 72, 264)]


def _whole(dev, n, L, R, inp, out, y, o):  # noqa: F811
    """(case, result)"""
    import torch

    c = Case(dev, _ids(n, L, n + R, run=1 if n < 200 else 60), inp, out, L, R, y, o, seed=n)
    g = torch.Generator(device=dev).manual_seed(n + R)
    k = torch.randint(1, 128, (3, n), generator=g, device=dev).double()
    at = [0, inp // 2 + 1, inp - 1]
    parts = [k[0] * 2.0 ** 14, k[1] * 2.0 ** 7, k[2]]
    c.x.zero_()
    for col, p in zip(at, parts):
        c.x[:, col] = p.bfloat16()
    sign = 1.0 - 2.0 * (torch.arange(R, device=dev) % 2)
    for col in at:
        c.a[:, :, col] = sign.bfloat16()
    c.scale = 2.0 ** (torch.arange(L, device=dev) % 3).float()
    # row o of B: one entry, 2^-(o mod 4), at rank (7 o + l) mod R
    rows = torch.arange(out, device=dev)
    c.b.zero_()
    factor = torch.zeros(n, out, dtype=torch.float64, device=dev)
    for l in range(L):
        i = (7 * rows + l) % R
        c.b[l, rows, i] = (2.0 ** -(rows % 4).float()).bfloat16()
        factor[c.ids == l] = 2.0 ** -(rows % 4).double() * sign[i].double() * float(c.scale[l])
    lead = parts[0] if y == "bf16" else parts[0] + parts[1]
    if c.y is not None:
        c.y = (-factor * lead[:, None]).to(c.y.dtype)
    want = factor * (parts[0] + parts[1] + parts[2])[:, None] + (0.0 if c.y is None else c.y.double())
    assert bool((want == want.float().double()).all())
    return c, want.float().to(c.out_type)


@pytest.mark.parametrize("n,L,R,inp,out", SIZES)
@pytest.mark.parametrize("y,o", [("bf16", "bf16"), ("fp32", "bf16"), (None, "bf16"), ("fp32", "fp32"), ("bf16", "fp32")])
def test_no_bit_of_v_is_lost(dev, n, L, R, inp, out, y, o):  # noqa: F811
    import torch

    c, want = _whole(dev, n, L, R, inp, out, y, o)
    got = c.run()
    assert torch.equal(got, want), int((got != want).sum())


@pytest.mark.parametrize("n,R", [(50, 32), (5000, 128)])
def test_in_place(dev, n, R):  # noqa: F811
    import torch

    c, want = _whole(dev, n, 3, R, 264, 136, "bf16", "bf16")
    assert torch.equal(c.run(out=c.y), want)
