"""The example layer against its plain float32 form.

Its own roundings to bfloat16 (each at most 2^-8 of a value): the gate-up rows, the
activation and the experts' rows, of which the output's relative distance sees less than their
sum, 4 * 2^-8 with the output's own; the router's gradient, a sum over the rows of products
with differences of nearly equal size, is allowed twice that."""

import os
import sys

import pytest

from gpu_util import show

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("tokens", [1, 5, 64, 700])
def test_moe_layer(tokens):
    import moe_layer
    show("example", tokens)
    y, grad = moe_layer.run(tokens)
    assert y <= 4 * 2.0 ** -8 and grad <= 8 * 2.0 ** -8
