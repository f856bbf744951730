"""GPU: adapters on batches around and above the 16384 tokens that one CTA groups, against the definition in 64 bits (and
its tolerance, as derived in test_gpu_lora.py)."""
import pytest

from test_gpu_lora import Case, _ids, dev  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [16384, 16385, 40000])
@pytest.mark.parametrize("L", [1, 7, 1024])
@pytest.mark.parametrize("run", [1, 300])
@pytest.mark.parametrize("y,o,R", [("bf16", "bf16", 16), ("fp32", "fp32", 128)])
def test_several_slices(dev, n, L, run, y, o, R):  # noqa: F811
    """In random order and in runs, tokens without an adapter in every slice."""
    from nvfp4_quantized_moe_topk_gb300 import api

    c = Case(dev, _ids(n, L, n + L, run), 72, 40, L, R, y, o, seed=L)
    c.check(c.run())
    assert api.lora_device_error() == 0


@pytest.mark.parametrize("L,run", [(7, 300), (1024, 1)])
def test_workspace_of_exactly_its_size(dev, L, run):  # noqa: F811
    """Of any content, and nothing beside it is written."""
    import torch

    from nvfp4_quantized_moe_topk_gb300 import api

    n = 40000
    c = Case(dev, _ids(n, L, 3, run), 72, 40, L, 16)
    want = c.run()
    size = api.load().moe_lora_workspace_bytes(n, L)
    room = torch.full((size + 512,), 0xFF, dtype=torch.uint8, device=dev)
    for fill in (0xFF, 0x11):
        room.fill_(fill)
        assert torch.equal(c.run(workspace=room[256:256 + size]), want)
        assert bool((room[:256] == fill).all()) and bool((room[256 + size:] == fill).all())


def test_one_adapter_or_none_in_whole_slices(dev):  # noqa: F811
    import torch

    n = 40000
    c = Case(dev, [2] * 16384 + [-1] * 16384 + [0] * (n - 32768), 72, 40, 4, 16, "fp32", "fp32")
    c.check(c.run())
    c.ids.fill_(-1)
    assert torch.equal(c.run(), c.y)
