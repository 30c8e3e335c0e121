"""The example's int4 quantiser: every weight comes back within its step (CPU only).

A code is off by half a step at most and the zero point by another half; the scale's rounding to
bfloat16 (2^-8 of it) moves the 15 steps of a group's range by 15 * 2^-8 of a step in all, also where
the last code is clamped."""

import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def weights(kind):
    g = torch.Generator().manual_seed(7)
    w = torch.rand((3, 5, 256), generator=g)
    return {"0.5 .. 1": 0.5 + 0.5 * w, "-1 .. -0.5": -0.5 - 0.5 * w, "-0.1 .. 2": 2.1 * w - 0.1, "-1 .. 1": 2 * w - 1,
            "far": 100.0 + w, "one value": torch.full_like(w, 0.7), "zeros": torch.zeros_like(w)}[kind]


@pytest.mark.parametrize("kind", ["0.5 .. 1", "-1 .. -0.5", "-0.1 .. 2", "-1 .. 1", "far", "one value", "zeros"])
@pytest.mark.parametrize("group", [32, 128, 256])
def test_weights_come_back_within_a_step(kind, group):
    import moe_layer
    w = weights(kind)
    packed, scale, zero = moe_layer.quantize_int4(w, group)
    back = moe_layer.dequantize_int4(packed, scale, zero, group)
    reach = w.unflatten(-1, (-1, group))
    step = (reach.amax(-1).clamp(min=0) - reach.amin(-1).clamp(max=0)) / 15.0
    assert torch.all((back - w).abs() <= (1.0 + 15 * 2.0 ** -8) * step.repeat_interleave(group, -1) + 1e-6)
    assert int(zero.max()) <= 15 and packed.shape == (3, 5, 128)
