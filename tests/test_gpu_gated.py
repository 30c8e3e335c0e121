"""GPU parity of the gated product and of the dense layer's gradients against the float64 oracle.

Tolerances, with u = 2^-24: a float32 sum of n products is off by at most (n + 8) u times the sum of
magnitudes B (8 for alpha, the addend and the matrix cores' own order), so both factors of a gated product
are off by t = (K + 8) u B; |act'| is at most 1.13, so the product by 1.13 t_g |u| + |act(g)| t_u + 1.13 t_g t_u,
and by (32 + 4 |z|) u of itself for the activation's own float32 steps, z its sigmoid's argument (its
rounding reaches the result |z|-fold).  An output rounded to bfloat16 adds half a step, 2^-8."""

import ctypes

import numpy as np
import pytest
import torch

import synth
from oracle import block as O
from oracle import formats
from gpu_util import DEV, show, to_dev_u8

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
ACTS = ["relu", "silu", "gelu_tanh"]
RATE = 2.0 * np.sqrt(2.0 / np.pi)


@pytest.fixture(scope="module")
def q():
    import weight_quantized_linear_amd as q
    return q


def f64(t):
    return t.double().cpu().numpy()


def random(rng, shape, dtype=torch.bfloat16, std=1.0):
    return torch.from_numpy(rng.normal(size=shape) * std).to(dtype).to(DEV)


def offset(t, by=1):
    """The same values at an address `by` elements behind an aligned one, poison around them."""
    flat = torch.full((t.numel() + by + 8,), 120, dtype=torch.uint8, device=DEV) if t.dtype == torch.uint8 else \
        torch.full((t.numel() + by + 8,), float("nan"), dtype=t.dtype, device=DEV)
    flat[by:by + t.numel()] = t.reshape(-1)
    return flat[by:by + t.numel()].view(t.shape)


def close(out, ref, tau, dtype):
    err = np.abs(f64(out) - ref)
    ok = err <= tau + HALF[dtype] * (np.abs(ref) + tau) + 2.0 ** -126
    if not ok.all():
        at = np.unravel_index(np.argmax(np.where(ok, 0, err / (tau + 1e-300))), ok.shape)
        print("worst at", at, "out", f64(out)[at], "ref", ref[at], "tau", tau[at], "bad", (~ok).sum(), "of", ok.size)
    return bool(ok.all())


def steepness(g, act):
    return {"relu": 0 * g, "silu": np.abs(g), "gelu_tanh": RATE * np.abs(g + 0.044715 * g ** 3)}[act]


def gated_tau(pre, bound, k, act):
    f = pre.shape[1] // 2
    t = (k + 8) * U * bound
    g, u, tg, tu = pre[:, :f], pre[:, f:], t[:, :f], t[:, f:]
    val = np.abs(O.activation(g, act)[0])
    return 1.13 * tg * np.abs(u) + val * tu + 1.13 * tg * tu + (32 + 4 * np.minimum(steepness(g, act), 1e3)) * U * val * np.abs(u)


def fp8_case(seed, rows, k):
    w, s = synth.fp8_weight((seed, rows, k), rows, k)
    return w, float(s)


def check_forward(q, rng, m, f, k, fp8, act, out_dtype, addend=None, odd=False):
    show("gated", m, f, k, fp8, act, out_dtype, addend, odd)
    x = random(rng, (m, k))
    alpha, alpha_up = 1.0, 1.0
    if fp8:
        codes, alpha = fp8_case(5, 2 * f, k)
        alpha_up = 1.5 * alpha
        w64, w = formats.e4m3_to_f64(codes), to_dev_u8(codes)
    else:
        w = random(rng, (2 * f, k), std=k ** -0.5)
        w64 = f64(w)
    c = random(rng, (m, 2 * f), addend, 0.5) if addend is not None else None
    if odd:
        w, x, c = offset(w), offset(x), None if c is None else offset(c)
    pre_dtype = torch.float32 if out_dtype == torch.float32 else torch.bfloat16
    room = torch.full((m * f + 16,), 7.0, dtype=out_dtype, device=DEV)
    start = 1 if odd else 8
    out = room[start:start + m * f].view(m, f)
    got, pre = q.gated_gemm(w, x, out=out, out_dtype=out_dtype, alpha=alpha, alpha_up=alpha_up, addend=c, activation=act,
                            return_pre=True, pre_dtype=pre_dtype)
    plain = q.gated_gemm(w, x, out_dtype=out_dtype, alpha=alpha, alpha_up=alpha_up, addend=c, activation=act)
    torch.cuda.synchronize()
    # alpha reaches the library as a float32
    ref, rpre, bound = O.gated(w64, f64(x), np.float32(alpha).astype(float), np.float32(alpha_up).astype(float),
                               None if c is None else f64(c), act)
    assert got.data_ptr() == out.data_ptr()
    assert bool((room[:start] == 7).all()) and bool((room[start + m * f:] == 7).all()), "writes outside out"
    assert close(got, ref, gated_tau(rpre, bound, k, act), out_dtype), "out"
    assert close(pre, rpre, (k + 8) * U * bound, pre_dtype), "pre"
    assert torch.equal(got, plain), "pre changes out"


SHAPES = [(1, 1, 1), (1, 16, 32), (2, 5, 7), (3, 33, 64), (4, 40, 100), (1, 130, 1023), (5, 64, 65), (16, 48, 256), (17, 31, 130),
          (33, 64, 64), (64, 128, 512), (65, 100, 96), (100, 257, 320), (130, 384, 1024), (300, 70, 2050),
          (260, 100, 133), (200, 4000, 192), (3, 40, 2056), (16, 24, 8192), (9, 17, 4104), (5, 70, 6000), (4, 21, 16400), (2, 9, 517)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,f,k", SHAPES)
def test_gated(q, fp8, out_dtype, m, f, k):
    check_forward(q, np.random.default_rng([1, m, f, k]), m, f, k, fp8, "silu", out_dtype)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("addend", [None, torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,f,k", [(1, 96, 256), (13, 64, 128), (40, 130, 192), (150, 256, 448)])
def test_gated_choices(q, act, addend, m, f, k):
    for fp8 in (False, True):
        check_forward(q, np.random.default_rng([2, m, f, k]), m, f, k, fp8, act, torch.bfloat16, addend)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("m,f,k", [(1, 48, 128), (16, 33, 64), (70, 128, 256), (260, 200, 128)])
def test_gated_off_alignment(q, fp8, m, f, k):
    check_forward(q, np.random.default_rng([3, m, f, k]), m, f, k, fp8, "silu", torch.bfloat16, torch.bfloat16, odd=True)


@pytest.mark.parametrize("m,f,k,fp8", [(1, 14336, 4096, True), (2, 4096, 14336, False), (16, 5504, 2048, False),
                                       (500, 2048, 4096, True), (700, 1408, 2048, False)])
def test_gated_large(q, m, f, k, fp8):
    check_forward(q, np.random.default_rng([4, m, f, k]), m, f, k, fp8, "silu", torch.bfloat16)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("m,f,k", [(17, 8300, 96), (64, 8256, 336), (33, 8193, 1040), (20, 8200, 128), (96, 130, 1040), (128, 200, 528),
                                   (65, 4099, 400), (64, 8192, 144)])
def test_gated_to_128_rows(q, fp8, m, f, k):
    """One tile of rows over wide and narrow layers, rows of k that end inside a strip."""
    check_forward(q, np.random.default_rng([12, m, f, k]), m, f, k, fp8, "silu", torch.bfloat16)
    check_forward(q, np.random.default_rng([13, m, f, k]), m, f, k, fp8, "relu", torch.float32, torch.bfloat16)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("addend", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,f,k", [(3, 37, 64), (7, 37001, 64), (16, 5504, 2064), (5, 1029, 4112), (13, 515, 8192)])
def test_addend_of_few_rows(q, fp8, addend, m, f, k):
    """Wide layers, of which a block has more tiles than it holds addends of, and every length of a row."""
    check_forward(q, np.random.default_rng([14, m, f, k]), m, f, k, fp8, "silu", torch.bfloat16, addend)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("grad_dtype,pre_dtype", [(torch.bfloat16, torch.float32), (torch.float32, torch.float32),
                                                  (torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("m,f", [(1, 1), (3, 7), (5, 64), (64, 257), (300, 1000)])
def test_activation_gradient(q, act, grad_dtype, pre_dtype, m, f):
    rng = np.random.default_rng([5, m, f])
    show("gated grad", act, grad_dtype, pre_dtype, m, f)
    pre = random(rng, (m, 2 * f), pre_dtype, 3.0)
    special = torch.tensor([0.0, -0.0, 90.0, -90.0, -100.0, 1e4, -1e4, 1e18, -1e18, 20.0], device=DEV).to(pre_dtype)
    n = min(10, f)
    pre[0, :n] = special[:n]
    dy = random(rng, (m, f), grad_dtype)
    w, x = random(rng, (2 * f, 4)), random(rng, (m, 4))
    got, dx, dw = q.gated_gemm_backward(dy, pre, w, x, activation=act, need_x=False, need_w=False)
    assert dx is None and dw is None and got.dtype == torch.bfloat16
    p, d = f64(pre), f64(dy)
    with np.errstate(over="ignore", invalid="ignore"):
        ref = O.gated_backward(d, np.where(np.abs(p) > 1e9, np.sign(p) * 1e3, p) if act == "gelu_tanh" else p, act)
    big = np.abs(p[:, :f]) > 1e9  # act is g or 0 there
    if act == "gelu_tanh":
        ref[:, f:][big] = (d * np.maximum(p[:, :f], 0))[big]
    g = p[:, :f]
    # the slope's two terms, each off by its own rounding
    z = np.minimum(steepness(g, act), 1e3)
    size = np.abs(d * p[:, f:]) * {"relu": 1.0, "silu": 1.0 + 0 * g, "gelu_tanh": 1.0 + 0 * g}[act]
    sig = 1.0 / (1.0 + np.exp(np.clip(-np.sign(g) * z, -500, 500)))
    rest = 1.0 / (1.0 + np.exp(np.clip(np.sign(g) * z, -500, 500)))
    slope = 0 * g if act == "relu" else sig * (1 + np.where(rest < 1e-30, 0, np.abs(g) * rest * (1 if act == "silu" else RATE * (1 + 0.14 * np.minimum(g * g, 1e6)))))
    tau = np.concatenate([size * slope, np.abs(ref[:, f:])], 1) * (48 + 4 * np.concatenate([z, z], 1)) * U
    assert close(got, ref, tau, torch.bfloat16)


LINEAR = [(1, 1, 1), (2, 3, 5), (16, 32, 64), (7, 130, 33), (64, 64, 64), (65, 127, 129), (128, 256, 64), (200, 96, 320), (333, 520, 264),
          (1, 512, 256), (31, 1000, 8), (256, 256, 512), (515, 264, 136)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", LINEAR)
@pytest.mark.parametrize("odd", [False, True])
def test_linear_gradients(q, dtype, m, n, k, odd):
    rng = np.random.default_rng([6, m, n, k])
    show("linear gradients", dtype, m, n, k, odd)
    dy, w, x = random(rng, (m, n)), random(rng, (n, k)), random(rng, (m, k))
    if odd:
        dy, w, x = offset(dy), offset(w), offset(x)
    d, w64, x64 = f64(dy), f64(w), f64(x)
    for call, other, ref, bound, terms in (
            (q.bf16_gemm_grad_x, w, d @ w64, np.abs(d) @ np.abs(w64), n),
            (q.bf16_gemm_grad_w, x, d.T @ x64, np.abs(d).T @ np.abs(x64), m)):
        room = torch.full((ref.size + 16,), 7.0, dtype=dtype, device=DEV)
        start = 1 if odd else 8
        out = room[start:start + ref.size].view(ref.shape)
        got = call(dy, other, out=out, out_dtype=dtype)
        assert got.data_ptr() == out.data_ptr()
        assert bool((room[:start] == 7).all()) and bool((room[start + ref.size:] == 7).all()), "writes outside out"
        assert close(got, ref, (terms + 8) * U * bound, dtype)


@pytest.mark.parametrize("m,n,k", [(2048, 2816, 1024), (1000, 4096, 1536), (4099, 520, 2048), (4096, 3000, 3328), (300, 9000, 264),
                                   (3000, 264, 520), (1500, 8256, 2040)])
def test_linear_gradients_large(q, m, n, k):
    test_linear_gradients(q, torch.bfloat16, m, n, k, False)


def test_linear_gradients_with_and_without_workspace(q):
    """Sums split over blocks and whole ones: both within the tolerance, and repeatable."""
    m, n, k = 200, 6000, 136
    rng = np.random.default_rng(8)
    dy, w, x = random(rng, (m, n)), random(rng, (n, k)), random(rng, (m, k))
    need = ctypes.c_int64(0)
    assert q.lib.qlinear_bf16_gemm_grad_workspace_size(m, n, k, ctypes.byref(need), None) == 0 and need.value > 0
    ref, bound = f64(dy) @ f64(w), np.abs(f64(dy)) @ np.abs(f64(w))
    for ws in (torch.empty(need.value, dtype=torch.uint8, device=DEV), torch.empty(16, dtype=torch.uint8, device=DEV)):
        got = q.bf16_gemm_grad_x(dy, w, out_dtype=torch.float32, workspace=ws)
        assert close(got, ref, (n + 8) * U * bound, torch.float32)
        assert torch.equal(got, q.bf16_gemm_grad_x(dy, w, out_dtype=torch.float32, workspace=ws))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,f,k", [(5, 24, 40), (130, 96, 64), (64, 129, 77)])
def test_gated_backward_is_the_forward_passs(q, act, m, f, k):
    """All gradients from the pre-activations that the forward call kept (float32), against the formula's: what
    is rounded on the way is dpre alone, 2^-8 of each value."""
    rng = np.random.default_rng([7, m, f, k])
    show("gated backward", act, m, f, k)
    w, x, dy = random(rng, (2 * f, k), std=k ** -0.5), random(rng, (m, k)), random(rng, (m, f))
    out, pre = q.gated_gemm(w, x, activation=act, return_pre=True)
    dpre, dx, dw = q.gated_gemm_backward(dy, pre, w, x, activation=act, grad_x_dtype=torch.float32,
                                         grad_w_dtype=torch.float32)
    assert pre.dtype == torch.float32
    w64, x64, d = f64(w), f64(x), f64(dpre)
    ref = O.gated_backward(f64(dy), f64(pre), act)
    assert np.all(np.abs(d - ref) <= 2.0 ** -8 * np.abs(ref) + 256 * U * np.abs(f64(pre)).max() * np.abs(f64(dy)).max())
    assert close(dx, d @ w64, (2 * f + 8) * U * (np.abs(d) @ np.abs(w64)), torch.float32)
    assert close(dw, d.T @ x64, (m + 8) * U * (np.abs(d).T @ np.abs(x64)), torch.float32)


def test_empty_and_not_finite(q):
    w, x = torch.ones((6, 8), dtype=torch.bfloat16, device=DEV), torch.ones((0, 8), dtype=torch.bfloat16, device=DEV)
    out, pre = q.gated_gemm(w, x, return_pre=True)
    assert out.shape == (0, 3) and pre.shape == (0, 6)
    dpre, dx, dw = q.gated_gemm_backward(out, pre, w, x)
    assert dpre.shape == (0, 6) and dx.shape == (0, 8) and not dw.any() and dw.shape == (6, 8)
    x = torch.ones((3, 8), dtype=torch.bfloat16, device=DEV)
    x[1, 2] = float("nan")
    y = q.gated_gemm(w, x)
    assert bool(y[1].isnan().all()) and bool(y[0::2].isfinite().all())
    x[1, 2] = float("inf")
    assert bool((q.gated_gemm(w, x)[1] == float("inf")).all())
