"""The feed-forward block's operators on operands of more than 4 GiB, where offsets in bytes pass 32 bits: the last
rows and columns, and samples between, against the float64 oracle on those alone.  Tolerances are those of
test_gpu_gated.py and test_gpu_block_norm.py."""

import numpy as np
import pytest
import torch

import test_gpu_block_norm as N
import test_gpu_gated as G
from oracle import block as O
from oracle import formats
from gpu_util import DEV, show

pytestmark = pytest.mark.gpu

GIB4 = 1 << 32


@pytest.fixture(scope="module")
def q():
    import weight_quantized_linear_amd as q
    return q


def normal(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device=DEV, dtype=dtype)


def sample(n, count=97):
    return torch.tensor(sorted(set(np.linspace(0, n - 1, count).astype(int).tolist() + [n - 2, n - 1, n // 2])), device=DEV)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("m", [1, 3, 13, 70])
def test_gated_with_large_weights(q, fp8, m):
    k = 8192
    f = (GIB4 // (k * (1 if fp8 else 2))) // 2 + 72
    assert 2 * f * k * (1 if fp8 else 2) > GIB4
    show("gated, large weights", m, f, k, fp8)
    gen = torch.Generator(device=DEV).manual_seed(1)
    w = torch.randint(0, 0x60, (2 * f, k), generator=gen, device=DEV, dtype=torch.uint8) if fp8 else normal(gen, 2 * f, k)
    x, at = normal(gen, m, k), sample(f)
    out, pre = q.gated_gemm(w, x, alpha=0.01, return_pre=True)
    part = torch.cat([w[at], w[at + f]])
    w64 = formats.e4m3_to_f64(part.cpu().numpy()) if fp8 else G.f64(part)
    alpha = float(np.float32(0.01))
    ref, rpre, bound = O.gated(w64, G.f64(x), alpha, alpha, None, "silu")
    assert G.close(pre[:, torch.cat([at, at + f])], rpre, (k + 8) * G.U * bound, torch.float32)
    assert G.close(out[:, at], ref, G.gated_tau(rpre, bound, k, "silu"), torch.bfloat16)


@pytest.mark.parametrize("k", [8192, 8195])
def test_gated_of_many_rows(q, k):
    f, m = 72, GIB4 // (2 * 8192) + 133
    show("gated, many rows", m, f, k)
    gen = torch.Generator(device=DEV).manual_seed(2)
    w, x, at = normal(gen, 2 * f, k), normal(gen, m, k), sample(m)
    out, pre = q.gated_gemm(w, x, alpha=0.01, return_pre=True)
    alpha = float(np.float32(0.01))
    ref, rpre, bound = O.gated(G.f64(w), G.f64(x[at]), alpha, alpha, None, "silu")
    assert G.close(pre[at], rpre, (k + 8) * G.U * bound, torch.float32)
    assert G.close(out[at], ref, G.gated_tau(rpre, bound, k, "silu"), torch.bfloat16)


@pytest.mark.parametrize("n", [8192, 8197])
def test_dense_gradients_of_many_rows(q, n):
    """grad_out of more than 4 GiB as the operand along and across the sum.  Values are -2 .. 2, so that all sums are
    exact: below 2^24."""
    m, k = GIB4 // (2 * 8192) + 133, 72
    assert 4 * m < 1 << 24
    show("dense gradients, many rows", m, n, k)
    gen = torch.Generator(device=DEV).manual_seed(3)
    dy, w, x = (torch.randint(-2, 3, s, generator=gen, device=DEV, dtype=torch.int8).to(torch.bfloat16) for s in ((m, n), (n, k), (m, k)))
    at, col = sample(m), sample(n, 33)
    dx = q.bf16_gemm_grad_x(dy, w, out_dtype=torch.float32)
    assert np.array_equal(G.f64(dx[at]), G.f64(dy[at]) @ G.f64(w))
    ref = G.f64(dy[:, col].t().contiguous()) @ G.f64(x)
    ws = torch.empty(16, dtype=torch.uint8, device=DEV)  # too small to split the sum
    for kw in (dict(), dict(workspace=ws)):
        assert np.array_equal(G.f64(q.bf16_gemm_grad_w(dy, x, out_dtype=torch.float32, **kw)[col]), ref)


def test_dense_gradients_of_large_results(q):
    m, n, k = 65536 + 72, 136, 32768 + 72
    assert m * k * 2 > GIB4
    show("dense gradients, large results", m, n, k)
    gen = torch.Generator(device=DEV).manual_seed(4)
    dy, w, at = normal(gen, m, n), normal(gen, n, k), sample(m)
    dx = q.bf16_gemm_grad_x(dy, w)
    d, w64 = G.f64(dy[at]), G.f64(w)
    assert G.close(dx[at], d @ w64, (n + 8) * G.U * (np.abs(d) @ np.abs(w64)), torch.bfloat16)
    del dx
    dy, x, at = normal(gen, n, m), normal(gen, n, k), sample(m)
    dw = q.bf16_gemm_grad_w(dy, x)
    d, x64 = G.f64(dy[:, at].t().contiguous()), G.f64(x)
    assert G.close(dw[at], d @ x64, (n + 8) * G.U * (np.abs(d) @ np.abs(x64)), torch.bfloat16)


@pytest.mark.parametrize("f", [4096, 4099])
def test_activation_gradient_of_many_rows(q, f):
    m = GIB4 // (4 * 4096) + 77
    show("activation gradient, many rows", m, f)
    gen = torch.Generator(device=DEV).manual_seed(5)
    pre, dy, at = normal(gen, m, 2 * f), normal(gen, m, f), sample(m)
    w, x = torch.zeros((2 * f, 1), dtype=torch.bfloat16, device=DEV), torch.zeros((m, 1), dtype=torch.bfloat16, device=DEV)
    got = q.gated_gemm_backward(dy, pre, w, x, need_x=False, need_w=False)[0]
    ref = O.gated_backward(G.f64(dy[at]), G.f64(pre[at]), "silu")
    # |act'| and its terms are below 1.13 and 2 at these gates, |act(g)| below |g|: 64 u of the factors' sizes covers all steps
    size = np.abs(G.f64(dy[at])) * (np.abs(G.f64(pre[at][:, f:])) + np.abs(G.f64(pre[at][:, :f])))
    assert G.close(got[at], ref, 64 * G.U * np.concatenate([size, size], 1), torch.bfloat16)


@pytest.mark.parametrize("h", [4096, 4091])
def test_norm_of_many_rows(q, h):
    t = GIB4 // (2 * 4096) + 4096 + 3
    show("norm, many rows", t, h)
    gen = torch.Generator(device=DEV).manual_seed(6)
    res, block, at = normal(gen, t, h), normal(gen, t, h), sample(t)
    w, wo = (normal(gen, h) for _ in range(2))
    y, r = q.block_norm(res, w, block=block, block_weight=wo)
    eps = float(np.float32(1e-6))
    ref, rr = O.norm(N.f64(res[at]), N.f64(w), N.f64(block[at]), N.f64(wo), None, 1.0, eps, lambda v: N.f64(r[at]))
    p = rr - N.f64(res[at])
    assert N.close("res", r[at], rr, 4 * N.U * np.abs(N.f64(res[at])) + (h / 2 + 20) * N.U * np.abs(p), N.B)
    assert N.close("out", y[at], ref, (h / 2 + 16) * N.U * np.abs(ref), N.B)
    # gradients come in for the sampled rows alone, so that the sums over rows have few terms
    dy, dr = torch.zeros_like(y), torch.zeros_like(res)
    dy[at], dr[at] = normal(gen, len(at), h), normal(gen, len(at), h)
    g = q.block_norm_backward(dy, dr, r, w, block=block, block_weight=wo)
    n = O.norm_backward(N.f64(dy[at]), N.f64(dr[at]), N.f64(r[at]), N.f64(w), N.f64(block[at]), N.f64(wo), None, 1.0, eps)
    row, col = (2 * h + 32) * N.U, (len(at) + 2 * h + 32) * N.U
    assert N.close("dres", g.residual[at], n["residual"], row * n["residual_bound"], N.B)
    assert N.close("dblock", g.block[at], n["block"], 2 * row * n["block_bound"], N.B)
    assert N.close("dw", g.weight, n["weight"], col * n["weight_bound"], N.B)
    assert N.close("dwo", g.block_weight, n["block_weight"], 2 * col * n["block_weight_bound"], N.B)
    rest = torch.ones(t, dtype=torch.bool, device=DEV)
    rest[at] = False
    assert not g.residual[rest].any() and not g.block[rest].any()
