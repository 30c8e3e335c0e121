"""Parity of the adapters where there are so many tiles that a block has a span of 1024 columns: each wave takes more than
one step of 64 of them.  Checks, oracle and tolerances are those of test_gpu_lora.py."""

import numpy as np
import pytest
import torch

import test_gpu_lora as L
from gpu_util import DEV

pytestmark = pytest.mark.gpu

B, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def q():
    import weight_quantized_linear_amd as q
    return q


@pytest.mark.parametrize("out_dtype", [B, F])
@pytest.mark.parametrize("base", [False, True])
@pytest.mark.parametrize("n,k,r", [(1100, 1035, 8), (1104, 1040, 33), (1100, 1035, 5)])
def test_adapters_of_many_tiles(q, out_dtype, base, n, k, r):
    """Spans of 1024 columns, of which a wave takes every fourth 64: more than one step of the second product's loop."""
    counts = [1] * 600
    assert len(counts) * -(-min(n, k) // 1024) >= 1024
    L.check(q, np.random.default_rng([24, n, r]), counts, 5, r, k, n, out_dtype, base)


@pytest.mark.parametrize("base", [False, True])
def test_adapters_of_many_tall_tiles(q, base):
    rng = np.random.default_rng(25)
    counts = rng.integers(40, 120, 200)
    L.check(q, rng, counts, 3, 16, 1035, 1104, B, base)
    L.check(q, rng, counts[:60], 3, 64, 1035, 1104, F, base)


def test_adapters_of_long_spans_in_place(q):
    rng = np.random.default_rng(26)
    off, ids = L.groups(rng, [1] * 600, 4)
    offs, idt = torch.from_numpy(off).to(DEV), torch.from_numpy(ids).to(DEV)
    for n, k in ((1100, 1035), (1104, 1040)):
        x, a, b = L.random(rng, (600, k)), L.random(rng, (4, 8, k)), L.random(rng, (4, n, 8))
        base, dy, dx0 = L.random(rng, (600, n)), L.random(rng, (600, n)), L.random(rng, (600, k))
        want, z = q.lora_gemm(x, a, b, offs, idt, base=base, return_z=True)
        got = base.clone()
        assert torch.equal(q.lora_gemm(x, a, b, offs, idt, base=got, out=got), want)
        wx, wa, wb = q.lora_gemm_backward(dy, x, z, a, b, offs, idt, base=dx0)
        buf = dx0.clone()
        gx, ga, gb = q.lora_gemm_backward(dy, x, z, a, b, offs, idt, base=buf, grad_x=buf)
        assert torch.equal(gx, wx) and torch.equal(ga, wa) and torch.equal(gb, wb)
