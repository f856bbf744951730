"""The Python calls of the operators around the layer: what is not a tensor, or not of the right form, is refused with the
framework's error, with and without a workspace of the caller's."""
import pytest

from nvfp4_quantized_moe_topk_gb300 import api


def _calls(bad):
    """(name, call) with `bad` in the place of each call's leading tensors."""
    import torch

    t = torch.zeros(4, 64, dtype=torch.bfloat16)
    yield "block_norm", lambda **kw: api.block_norm(bad)
    yield "block_norm_backward", lambda **kw: api.block_norm_backward(bad, None, None, **kw)
    yield "block_norm_backward u", lambda **kw: api.block_norm_backward(None, None, bad, **kw)
    yield "balance_loss", lambda **kw: api.balance_loss(bad, None, bad, bad, bad, bad, bad, coef=1.0, **kw)
    yield "balance_loss offsets", lambda **kw: api.balance_loss(t, None, t, t, t, t, t, coef=1.0, seq_offsets=bad, **kw)
    yield "router_backward", lambda **kw: api.router_backward(bad, None, bad, None, None, None, None, bad, coef=1.0, **kw)
    yield "lora_apply x", lambda **kw: api.lora_apply(bad, t, t, t, t, t, **kw)
    yield "lora_apply a", lambda **kw: api.lora_apply(t, t, bad, t, t, t, **kw)


@pytest.mark.parametrize("bad", [[[1.0, 2.0]], "x", 3.0, object()], ids=["list", "text", "number", "object"])
@pytest.mark.parametrize("given", [False, True])
def test_what_is_not_a_tensor(bad, given):
    import torch

    kw = dict(workspace=torch.empty(64, dtype=torch.uint8)) if given else {}
    for name, call in _calls(bad):
        with pytest.raises(api.MoeError) as e:
            call(**({} if name == "block_norm" else kw))
        assert e.value.status == 1, name


@pytest.mark.gpu
def test_tensors_of_other_dimensions():
    """Before the workspace is made for them."""
    import torch

    dev = torch.device("cuda:0")
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=dev)
    ids = torch.zeros(4, dtype=torch.int32, device=dev)
    scalar = torch.zeros((), dtype=torch.bfloat16, device=dev)
    for a in (scalar, x, None):
        with pytest.raises(api.MoeError):
            api.lora_apply(x, ids, a, x[None], None, x)
    logits = torch.zeros(4, 8, device=dev)
    for offsets in (torch.zeros((), dtype=torch.int32, device=dev), ids[:0], ids[None]):
        with pytest.raises(api.MoeError):
            api.balance_loss(logits, None, ids[:, None], logits[0, :1], ids, logits, ids, coef=1.0, seq_offsets=offsets)


@pytest.mark.gpu
def test_stream_that_is_no_handle():
    """Nothing is enqueued on another stream in its place."""
    import torch

    dev = torch.device("cuda:0")
    r = torch.ones(4, 64, dtype=torch.bfloat16, device=dev)
    w, x = torch.ones(64, dtype=torch.bfloat16, device=dev), torch.full_like(r, 7.0)
    for stream in (1 << 70, "main", object()):
        with pytest.raises((api.MoeError, TypeError, OverflowError, AttributeError)):
            api.block_norm(r, pre_weight=w, x_out=x, stream=stream)
    torch.cuda.synchronize()
    assert bool((x == 7.0).all())
