"""Rotations by small angles, where a pair's first member is zero and its output is the sine alone.

The angle is within 2^-54 turns times the position of the exact one and 2^-24 of itself; sine and cosine are within 2 u of
their argument's (test_gpu_qk), the products and the scale 3 u more: 16 u of the value allow for all but the turns."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from nvfp4_quantized_moe_topk_gb300 import api  # noqa: E402

DEV, D, U = "cuda", torch.float64, 2.0 ** -24


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("backward", [False, True])
def test_the_sine_of_a_small_angle(interleaved, backward):
    pairs = 64
    freq = torch.logspace(0, -9, pairs, dtype=D, device=DEV).float()
    pos = torch.tensor([0, 1, -1, 2, 3, -7, 100, 4095, -4096, 131072, 2 ** 20 + 1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32,
                       device=DEV)
    n = pos.numel()
    q = torch.zeros(n, 1, 2 * pairs, device=DEV)
    second = q[..., 1::2] if interleaved else q[..., pairs:]
    second.fill_(1.0)
    out = torch.empty_like(q)
    if backward:
        api.qk_norm_rope_backward(q, None, q, None, out, None, pos, freq, pairs_interleaved=interleaved)
    else:
        api.qk_norm_rope(q, None, out, None, pos, freq, pairs_interleaved=interleaved)
    angle = pos.to(D)[:, None] * freq.to(D)
    sign = 1 if backward else -1
    got_s, got_c = (out[:, 0, 0::2], out[:, 0, 1::2]) if interleaved else (out[:, 0, :pairs], out[:, 0, pairs:])
    turns = 2 * math.pi * 2.0 ** -54 * pos.to(D).abs()[:, None]
    own = angle.abs() * 2.0 ** -52  # of the reference's own angle in 64 bits
    assert bool(((got_s.to(D) - sign * torch.sin(angle)).abs() <= 16 * U * torch.sin(angle).abs() + turns + own
                 + 4 * U * (angle.abs() > 1.5)).all())
    assert bool(((got_c.to(D) - torch.cos(angle)).abs() <= 16 * U + turns + own).all())
