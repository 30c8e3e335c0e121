"""The gated activation at gates whose sigmoid is below float32's smallest normal number
while the results are not, against the float64 oracle.

With u = 2^-24: exp(-|g| / 2) is off by 3 u, used twice; 1 / (1 + exp(-|g|)) by 6 u at most, of which
1 + g sigmoid(-g) sees as much again; five products add one each: 24 u in all, relative to the sum
of magnitudes.  A bfloat16 output adds half a step.  Results below the smallest normal
number (2^-126) are free."""

import numpy as np
import pytest
import torch

from oracle import moe as O
from gpu_util import DEV, show

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
TINY = 2.0 ** -126


@pytest.fixture(scope="module")
def q():
    import weight_quantized_linear_amd as q
    return q


def operands(gates, ups, grads, dtype):
    """Every combination in one row, and one more column so that it ends off 16 bytes."""
    g, u, d = (v.reshape(-1) for v in np.meshgrid(gates, ups, grads, indexing="ij"))
    g, u, d = (np.append(v, 0.5) for v in (g, u, d))
    x = torch.from_numpy(np.stack([np.concatenate([g, u])] * 3)).to(dtype).to(DEV)
    return x, torch.from_numpy(np.stack([d] * 3)).to(dtype).to(DEV)


def check(q, x, dy, dtype):
    x64, d64 = x.double().cpu().numpy(), dy.double().cpu().numpy()
    ref = O.swiglu(x64)
    tau = 24 * U * np.abs(ref)
    err = np.abs(q.swiglu(x).double().cpu().numpy() - ref)
    assert np.all(err <= tau + HALF[dtype] * (np.abs(ref) + tau) + TINY)
    ref, bound = O.swiglu_backward(d64, x64)
    tau = 24 * U * bound
    err = np.abs(q.swiglu_backward(dy, x).double().cpu().numpy() - ref)
    assert np.all(err <= tau + HALF[dtype] * (np.abs(ref) + tau) + TINY)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_subnormal_sigmoid_keeps_its_products(q, dtype):
    show("swiglu subnormal sigmoid", dtype)
    x, dy = operands([-86.5, -87.5, -88.0, -90.0, -100.0, -103.5, -120.0, -150.0, -170.0], [1.0, -1e10, 1e20, 1e30],
                     [1.0, 1e10, -1e18], dtype)
    check(q, x, dy, dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_an_overflowing_product_of_the_factors_is_not_formed(q, dtype):
    """dy u passes float32's range, their product with the sigmoid does not; gates 0 and above keep small factors."""
    show("swiglu large factors", dtype)
    x, dy = operands([-60.0, -100.0, -150.0, -170.0], [1e25, -1e25], [1e25, -1e22], dtype)
    check(q, x, dy, dtype)
    x, dy = operands([-30.0, -1.0, -1e-30, 0.0, 1e-30, 1.0, 30.0, 100.0], [1e15, -1e-15], [1e15, -1e-15], dtype)
    check(q, x, dy, dtype)


def test_infinite_and_nan_gates(q):
    """+inf passes as the formula has it (1 + exp(-inf) = 1); -inf / inf and NaN are NaN; their neighbours stay."""
    inf, nan = float("inf"), float("nan")
    x = torch.tensor([[inf, -inf, nan, 1.0, 2.0, 2.0, 2.0, 2.0]], device=DEV)
    show("swiglu infinite gates")
    y = q.swiglu(x).cpu()[0]
    assert y[0] == inf and torch.isnan(y[1]) and torch.isnan(y[2]) and abs(float(y[3]) - 2 * 0.7310585786) < 1e-5
