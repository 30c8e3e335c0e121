"""The norm at the largest magnitudes that its rows may have: 2^56 at any width, where the sum of 2^14 squares is 2^126.
Tolerances as in test_gpu_block_norm.py."""

import numpy as np
import pytest
import torch

import test_gpu_block_norm as N
from oracle import block as O
from gpu_util import DEV, show

pytestmark = pytest.mark.gpu

TOP = 2.0 ** 56


@pytest.mark.parametrize("h", [1, 2, 5, 4096, 16381, 16384])
@pytest.mark.parametrize("types", [(N.B, N.B, N.B), (N.F, N.F, N.F)])
def test_rows_at_the_top_of_the_range(h, types):
    import weight_quantized_linear_amd as q
    rt, bt, pt = types
    show("norm range", h, types)
    rng = np.random.default_rng(h)

    def large(dtype, top):
        """Magnitudes within one binary order below `top`, and not above it when rounded."""
        v = rng.uniform(0.5, 0.99, (3, h)) * rng.choice([-1.0, 1.0], (3, h)) * top
        return torch.from_numpy(v).to(dtype).to(DEV)

    # residual_out = residual / 2 + the normed block, which is about its weight: both terms stay in the range
    res, block, w = large(rt, TOP), large(bt, TOP), torch.ones(h, dtype=pt, device=DEV)
    wo = torch.from_numpy(rng.uniform(0.5, 1.0, h)).to(pt).to(DEV)
    y, r2 = q.block_norm(res, w, block=block, block_weight=wo, residual_scale=0.5)
    ref, rr = O.norm(N.f64(res), N.f64(w), N.f64(block), N.f64(wo), None, 0.5, float(np.float32(1e-6)), lambda v: N.f64(r2))
    assert N.close("res", r2, rr, (h / 2 + 24) * N.U * np.abs(rr), rt)
    assert N.close("out", y, ref, (h / 2 + 16) * N.U * np.abs(ref), bt)
    plain, _ = q.block_norm(res, w, out_dtype=bt)
    ref, _ = O.norm(N.f64(res), N.f64(w), None, None, None, 1.0, float(np.float32(1e-6)), lambda v: v)
    assert N.close("plain", plain, ref, (h / 2 + 16) * N.U * np.abs(ref), bt)

    dy, dr = large(bt, 1.0), large(rt, 2.0 ** -56)
    g = q.block_norm_backward(dy, dr, r2, w, block=block, block_weight=wo, residual_scale=0.5)
    n = O.norm_backward(N.f64(dy), N.f64(dr), N.f64(r2), N.f64(w), N.f64(block), N.f64(wo), None, 0.5, float(np.float32(1e-6)))
    row, col = (2 * h + 32) * N.U, (3 + 2 * h + 32) * N.U
    assert N.close("dres", g.residual, n["residual"], row * n["residual_bound"], rt)
    assert N.close("dw", g.weight, n["weight"], col * n["weight_bound"], pt)
    assert N.close("dblock", g.block, n["block"], 2 * row * n["block_bound"], bt)
    assert N.close("dwo", g.block_weight, n["block_weight"], 2 * col * n["block_weight_bound"], pt)
