"""Adapters over more rows than one launch has threads for (T up to 2^30 is allowed).

Rows are zeros but for a few, so the results are zeros but for theirs and the parameters' gradients are sums over
those few: the oracle takes them alone.  Tolerances as in test_gpu_lora.py: z K + 8 u of the sum of magnitudes
(u = 2^-24), out K + 3 R + 32 u and 2^-16 of it and half a bfloat16 step, dA and dB the same with the rows that count."""

import numpy as np
import pytest
import torch

from oracle import block as O
from gpu_util import DEV, show

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def q():
    import weight_quantized_linear_amd as q
    return q


def test_rows_past_a_launch(q):
    t, k, n, r = (1 << 29) + 77, 8, 8, 1
    show("lora", t, k, n, r)
    rng = np.random.default_rng(1)
    at = np.array([0, 1, 33, (1 << 28) + 5, (1 << 29) - 1, 1 << 29, (1 << 29) + 64, t - 1])
    rows = torch.from_numpy(at).to(DEV)

    def few(width):
        v = torch.from_numpy(rng.normal(size=(len(at), width))).to(torch.bfloat16).to(DEV)
        full = torch.zeros((t, width), dtype=torch.bfloat16, device=DEV)
        full[rows] = v
        return full, v.double().cpu().numpy()

    x, x64 = few(k)
    dy, dy64 = few(n)
    a, b = (torch.from_numpy(rng.normal(size=s)).to(torch.bfloat16).to(DEV) for s in ((1, r, k), (1, n, r)))
    a64, b64 = a.double().cpu().numpy(), b.double().cpu().numpy()
    off, ids = torch.tensor([0, t], dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    small, one = [0, len(at)], np.ones(1)
    out, z = q.lora_gemm(x, a, b, off, ids, return_z=True)
    ref, rz, bound, zb, _ = O.lora(x64, a64, b64, small, [0], one, None, n)
    assert np.all(np.abs(z[rows].double().cpu().numpy() - rz) <= (k + 9) * U * zb)
    tau = ((k + 3 * r + 32) * U + 2.0 ** -16) * bound
    assert np.all(np.abs(out[rows].double().cpu().numpy() - ref) <= tau + 2.0 ** -8 * (np.abs(ref) + tau))
    out[rows] = 0
    assert int(torch.count_nonzero(out)) == 0 and int(torch.count_nonzero(z)) == len(at)
    del out
    dx, da, db = q.lora_gemm_backward(dy, x, z, a, b, off, ids)
    rx, ra, rb, xb, ab, bb = O.lora_backward(dy64, x64, z[rows].double().cpu().numpy(), a64, b64, small, [0], one, None)
    tau = ((n + 3 * r + 32) * U + 2.0 ** -16) * xb
    assert np.all(np.abs(dx[rows].double().cpu().numpy() - rx) <= tau + 2.0 ** -8 * (np.abs(rx) + tau))
    dx[rows] = 0
    assert int(torch.count_nonzero(dx)) == 0
    terms = 3 * len(at)  # zeros add nothing
    assert np.all(np.abs(da.double().cpu().numpy() - ra) <= (n + terms + 33) * U * ab)
    assert np.all(np.abs(db.double().cpu().numpy() - rb) <= (terms + 33) * U * bb)
