"""The whole layer's logits from an fp32 router weight of any value: finite ones up to the largest, and infinities.

A weight w above bf16's largest value (2^128 - 2^119.4) is one that no bf16 term may be rounded up from.  The columns of x that
meet it hold 2^-100 or 0, so that w x stays finite; tolerance as in test_gpu_layer_forward: (H / 16 + 16) 2^-22 of
sum |x w|, three times as many steps for three terms."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from nvfp4_quantized_moe_topk_gb300 import api  # noqa: E402
from test_gpu_layer_forward import D, Layer  # noqa: E402

MOST = torch.finfo(torch.float32).max


def _layer():
    layer = Layer(router="fp32", S=1)
    layer.router[3, 10], layer.router[4, 11], layer.router[5, 12] = MOST, -MOST, 3.395e38
    layer.router[6, 13] = float(torch.finfo(torch.bfloat16).max)
    return layer


@pytest.mark.parametrize("n", [1, 5, 40, 64, 100])
def test_the_largest_weights(n):
    layer = _layer()
    x = layer.randn(n, layer.H).to(torch.bfloat16)
    x[:, 10:14] = 2.0 ** -100
    x[0, 10:14] = 0
    _, ids, weights, logits = layer.call(x, bias=False)
    xd, r = x.to(D), layer.router.to(D)
    want = xd @ r.t()
    bound = 3 * (layer.H / 16 + 16) * 2.0 ** -22 * (xd.abs() @ r.abs().t())
    assert bool(logits.isfinite().all()) and bool(((logits.to(D) - want).abs() <= bound).all())
    want_ids, want_w = torch.empty_like(ids), torch.empty_like(weights)
    api.router_topk(logits, None, want_ids, want_w)
    assert torch.equal(ids, want_ids) and torch.equal(weights, want_w)


@pytest.mark.parametrize("n", [1, 5, 40, 64, 100])
def test_an_infinite_weight_gives_infinite_logits(n):
    layer = Layer(router="fp32", S=1)
    x = layer.randn(n, layer.H).to(torch.bfloat16)
    x[:, 20] = 0.5
    x[0, 20] = -0.5
    layer.router[7, 20], layer.router[8, 21] = float("inf"), float("nan")
    logits = layer.call(x, bias=False)[3]
    assert bool((logits[1:, 7] == float("inf")).all()) and float(logits[0, 7]) == float("-inf")
    assert bool(logits[:, 8].isnan().all())
    rest = [e for e in range(layer.E) if e not in (7, 8)]
    assert bool(logits[:, rest].isfinite().all())
