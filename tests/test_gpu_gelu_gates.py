"""The tanh GELU's gradient at gates so large that their product with the slope's steps passes float32's range.

From |g| = 32 on sigmoid(z) is 1 or 0 to more than 400 digits, so d act(g) / dg is 1 or 0 and act(g) is g or 0: the
gradients are [dy u, dy g] for gates above and [0, 0] for gates below.  Of the factors 1 is exact, so each result is
two or three float32 products of the values, 4 u of itself at most (u = 2^-24), and rounded to bfloat16: half a step, 2^-8."""

import pytest
import torch

from gpu_util import DEV, show

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def q():
    import weight_quantized_linear_amd as q
    return q


@pytest.mark.parametrize("pre_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("grad_dtype", [torch.float32, torch.bfloat16])
def test_gelu_gradient_of_large_gates(q, pre_dtype, grad_dtype):
    show("gelu gradient, large gates", pre_dtype, grad_dtype)
    gates = torch.tensor([40.0, 1e10, 1e30, 1.2e36, 1.6e36, 1e37, 3.3e38], device=DEV)
    gates = torch.cat([gates, -gates])
    g, u, d = (v.reshape(-1) for v in torch.meshgrid(gates, torch.tensor([1.0, -2.5, 0.0], device=DEV),
                                                     torch.tensor([1.0, -0.5], device=DEV), indexing="ij"))
    pre = torch.cat([g, u]).to(pre_dtype).repeat(2, 1)
    dy = d.to(grad_dtype).repeat(2, 1)
    f = dy.shape[1]
    w, x = torch.zeros((2 * f, 8), dtype=torch.bfloat16, device=DEV), torch.zeros((2, 8), dtype=torch.bfloat16, device=DEV)
    got = q.gated_gemm_backward(dy, pre, w, x, activation="gelu_tanh", need_x=False, need_w=False)[0].double()
    g, u, d = pre[:, :f].double(), pre[:, f:].double(), dy.double()
    want = torch.cat([d * u * (g > 0), d * g.clamp(min=0.0)], 1)
    assert bool(got.isfinite().all())
    assert bool(((got - want).abs() <= (4 * U + 2.0 ** -8) * want.abs()).all())


def test_gelu_gradient_of_a_nan_gate(q):
    pre = torch.ones((1, 16), device=DEV)
    pre[0, 3] = float("nan")
    w, x = torch.zeros((16, 8), dtype=torch.bfloat16, device=DEV), torch.zeros((1, 8), dtype=torch.bfloat16, device=DEV)
    show("gelu gradient, NaN gate")
    got = q.gated_gemm_backward(torch.ones((1, 8), device=DEV), pre, w, x, activation="gelu_tanh", need_x=False, need_w=False)[0]
    assert got.isnan().nonzero()[:, 1].tolist() == [3, 11]
