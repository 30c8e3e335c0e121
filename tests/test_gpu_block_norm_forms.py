"""The block norm's forward forms for large calls: results past the caches (above 160 MiB moved), and more rows than
one turn of the grid has.  Oracle and tolerances are those of test_gpu_block_norm.py."""

import numpy as np
import pytest
import torch

import test_gpu_block_norm as N
from oracle import block as O
from gpu_util import DEV, show

pytestmark = pytest.mark.gpu

B, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def q():
    import weight_quantized_linear_amd as q
    return q


def rows_of_norm(q, t, h, types, post, gates, in_place, take):
    """The forward call on t rows, of which the oracle has those in `take`; everything is compared on the device
    with the same rows in a call of their own, which takes another form."""
    rt, bt, pt = types
    show("norm rows", t, h, types, post, gates, in_place)
    g = torch.Generator(device=DEV).manual_seed(t + h)
    res, block = torch.randn((t, h), generator=g, device=DEV).to(rt), torch.randn((t, h), generator=g, device=DEV).to(bt)
    w = (torch.randn(h, generator=g, device=DEV) * 0.3 + 1).to(pt)
    wo = (torch.randn(h, generator=g, device=DEV) * 0.3 + 1).to(pt) if post else None
    gate = torch.randn((gates, h), generator=g, device=DEV).to(pt) if gates else None
    kept = res[take].clone()
    room = torch.full((t + 2, h), 7.0, dtype=bt, device=DEV)
    y, r2 = q.block_norm(res, w, block=block, block_weight=wo, gate=gate, residual_scale=0.5, out=room[1:t + 1],
                         residual_out=res if in_place else None)
    assert bool((room[0] == 7).all()) and bool((room[t + 1] == 7).all()), "writes outside out"
    own = None if gate is None else gate[take * gates // t].contiguous()
    y2, r3 = q.block_norm(kept, w, block=block[take].contiguous(), block_weight=wo, gate=own, residual_scale=0.5)
    assert torch.equal(y[take], y2) and torch.equal(r2[take], r3)
    ref, rr = O.norm(N.f64(kept), N.f64(w), N.f64(block[take]), N.f64(wo), N.f64(own), 0.5, float(np.float32(1e-6)),
                     lambda v: N.f64(r3))
    p = rr - 0.5 * N.f64(kept)
    assert N.close("res", r3, rr, 4 * N.U * np.abs(0.5 * N.f64(kept)) + (h / 2 + 20) * N.U * np.abs(p), rt)
    assert N.close("out", y2, ref, (h / 2 + 16) * N.U * np.abs(ref), bt)


@pytest.mark.parametrize("types,t,h", [((B, B, B), 10400, 2048), ((B, B, F), 20500, 1027), ((F, B, B), 3600, 4096),
                                       ((F, F, F), 1300, 8199), ((F, B, F), 28000, 511)])
def test_norm_past_the_caches(q, types, t, h):
    """Results of more than 160 MiB moved are stored past the caches."""
    size = {B: 2, F: 4}
    assert t * h * 2 * (size[types[0]] + size[types[1]]) > 160 << 20
    take = torch.arange(0, t, 7, device=DEV)
    for post, gates, in_place in ((True, 1, False), (False, 4, True)):
        rows_of_norm(q, t, h, types, post, gates if t % gates == 0 else 1, in_place, take)


@pytest.mark.parametrize("t,h,types", [(65536 + 3, 1032, (B, B, B)), (2 * 65536 + 77, 515, (F, B, F)), (4 * 65536 + 131, 24, (B, B, F)),
                                       (2 * 65536 + 5, 1029, (B, B, B))])
@pytest.mark.parametrize("post", [False, True])
def test_norm_of_more_rows_than_the_grid(q, t, h, types, post):
    """A block's second turn, in which its sums go to LDS words that the first may still be reading."""
    per = 1 if h > 1024 else 2 if h > 512 else 4
    assert -(-t // per) > 65536
    take = torch.cat([torch.arange(0, t, 61, device=DEV), torch.arange(65536 * per - 9, t, device=DEV)]).unique()
    rows_of_norm(q, t, h, types, post, 1, True, take)
