"""The whole layer where a handle runs more than 64 tokens as one launch: the picks come from a kernel of their own, and
the experts stay whole however many tokens take them.  Tolerances: test_gpu_layer_forward."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from test_gpu_layer_forward import Layer  # noqa: E402


@pytest.mark.parametrize("n", [65, 70, 100, 128])
@pytest.mark.parametrize("kw", [dict(S=1), dict(S=2, gated=True), dict(S=2, k=3, E=40, router="fp32"), dict(S=0, k=5)])
def test_more_tokens_as_one_launch_than_the_router_routes(n, kw):
    layer = Layer(single=200, **kw)
    layer.check(n)


@pytest.mark.parametrize("kw", [dict(S=1), dict(S=2, gated=True)])
def test_parts_of_an_earlier_batch_are_not_taken(kw):
    """Batches whose experts are cut into parts, of several sizes, before and after one whose experts are not."""
    layer = Layer(single=200, **kw)
    layer.bias[: layer.k - 1] += 4.0  # experts that most tokens pick
    for n in (64, 9, 33, 100, 17, 70, 1, 128, 40):
        layer.check(n)


def test_graph_and_same_bits():
    layer = Layer(single=200, S=2)
    x = layer.randn(100, layer.H).to(torch.bfloat16)
    first = layer.call(x)
    layer.call(x[:40].contiguous())
    for a, b in zip(first, layer.call(x)):
        assert torch.equal(a, b)
    graph, dst = torch.cuda.CUDAGraph(), torch.empty_like(x)
    with torch.cuda.graph(graph):
        layer.layer.layer_forward(x, layer.router, dst, None, layer.bias, shared_experts=2)
    for _ in range(2):
        graph.replay()
    assert torch.equal(dst, first[0])


def test_the_picks_are_the_forward_s():
    """Without shared experts one launch takes the same picks as moe_nvfp4_forward, onto the same residual: the same bits."""
    layer = Layer(S=0, single=200)
    x, res = layer.randn(100, 256).to(torch.bfloat16), layer.randn(100, 256).to(torch.bfloat16)
    dst, ids, weights, _ = layer.call(x, res)
    want = res.clone()
    layer.layer.forward(x, ids, weights, want)
    assert torch.equal(dst, want)
