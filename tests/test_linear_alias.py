"""The projections' arrays that may not be one another, and more tokens than they count, without a GPU (no accepted call is
made here: the addresses are not memory)."""
import pytest

from test_linear_abi import A, args, grads, lib  # noqa: F401

OWN = dict(z=16 * A, res=17 * A, bias=18 * A)


@pytest.mark.parametrize("kw", [dict(bias=2 * A), dict(bias=16 * A), dict(bias=2 * A, z=0)])
def test_no_output_is_the_bias(lib, kw):  # noqa: F811
    """The bias is read by tiles that follow others' stores."""
    assert lib.moe_linear(args(**dict(OWN, **kw)), None) == 1


@pytest.mark.parametrize("gk", [dict(dx=4 * A), dict(db=4 * A), dict(db=3 * A)])
def test_no_gradient_is_another(lib, gk):  # noqa: F811
    assert lib.moe_linear_backward(args(**OWN), grads(**dict(dict(dy=19 * A), **gk)), 8 * A, 1 << 40, None) == 1


@pytest.mark.parametrize("at", [19 * A, 7 * A, 6 * A, 16 * A, 3 * A, 4 * A, 5 * A])
def test_the_workspace_is_its_own(lib, at):  # noqa: F811
    """d_out, x, weight and z are read after the workspace has been written."""
    assert lib.moe_linear_backward(args(act=1, **OWN), grads(dy=19 * A), at, 1 << 40, None) == 1


@pytest.mark.parametrize("n", [(1 << 31) - 1023, (1 << 31) - 1])
def test_tokens_that_32_bits_do_not_count(lib, n):  # noqa: F811
    """The last rows' numbers, rounded up to a tile or a turn, would pass 2^31."""
    assert lib.moe_linear(args(n=n, **OWN), None) == 2
    assert lib.moe_linear_backward(args(n=n, **OWN), grads(dy=19 * A), 8 * A, 1 << 60, None) == 2
