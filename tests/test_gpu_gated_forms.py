"""Parity of the gated product and of the dense layer's gradients in the tiles that they take at sizes of real use.
Checks, oracle and tolerances are those of test_gpu_gated.py; sizes are small ones for which the launcher takes the
tile, and each test asserts the choice, by the launcher's rule on this card's CUs."""

import numpy as np
import pytest
import torch

import test_gpu_gated as G
from gpu_util import DEV, show

pytestmark = pytest.mark.gpu

B, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def q():
    import weight_quantized_linear_amd as q
    return q


def cus():
    return torch.cuda.get_device_properties(0).multi_processor_count


def tiles(m, n, bm, bn):
    return -(-m // bm) * -(-n // bn)


def rounds(m, n, bm, bn, slots):
    return -(-tiles(m, n, bm, bn) // slots)


# ---------------------------------------------------------------- gated product


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("out_dtype,addend,act", [(B, None, "silu"), (F, B, "gelu_tanh"), (B, F, "relu")])
@pytest.mark.parametrize("m,f,k", [(490, 14344, 144), (2050, 2824, 80), (2050, 2817, 208)])
def test_gated_tile_of_a_whole_cu(q, fp8, out_dtype, addend, act, m, f, k):
    """256 rows x 128 columns, eight waves; the last tiles of rows, columns and k are parts."""
    assert 1.75 * rounds(m, f, 256, 128, cus()) <= 1.05 * rounds(m, f, 128, 64, 2 * cus())
    G.check_forward(q, np.random.default_rng([20, m, f, k]), m, f, k, fp8, act, out_dtype, addend)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("out_dtype,addend", [(B, None), (F, B)])
@pytest.mark.parametrize("m,f,k,odd", [(515, 4133, 67, False), (260, 5500, 72, True), (700, 2817, 131, True)])
def test_gated_staged_tile_of_128_rows(q, fp8, out_dtype, addend, m, f, k, odd):
    assert tiles(m, f, 128, 64) > cus()
    G.check_forward(q, np.random.default_rng([21, m, f, k]), m, f, k, fp8, "silu", out_dtype, addend, odd=odd)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("m,f,k,odd", [(1, 21, 96, False), (2, 21, 100, False), (4, 21, 99, False), (5, 40, 96, False), (16, 40, 4096, False),
                                       (20, 8192, 256, False), (20, 40, 160, False), (100, 40, 160, False), (150, 72, 160, False),
                                       (490, 14344, 32, False), (20, 40, 101, False), (515, 4133, 67, False), (9, 40, 5, False)])
def test_gated_not_finite_stays_in_its_row_and_column(q, fp8, m, f, k, odd):
    """Every form: a NaN in a row of x, in a gate row and in an up row of w reach that row and those columns alone."""
    show("gated not finite", m, f, k, fp8)
    rng = np.random.default_rng([22, m, f, k])
    x = G.random(rng, (m, k))
    w = torch.from_numpy(rng.integers(0, 0x60, (2 * f, k)).astype(np.uint8)).to(DEV) if fp8 else G.random(rng, (2 * f, k))
    w[f - 3, k - 1] = 0xFF if fp8 else float("nan")
    w[f + 2, 0] = 0x7F if fp8 else float("nan")
    if m > 1:
        x[m - 2, k // 2] = float("nan")
    out, pre = q.gated_gemm(w, x, return_pre=True)
    want = torch.zeros((m, 2 * f), dtype=torch.bool, device=DEV)
    want[:, f - 3] = want[:, f + 2] = True
    if m > 1:
        want[m - 2] = True
    assert torch.equal(pre.isnan(), want) and torch.equal(out.isnan(), want[:, :f] | want[:, f:])


# ---------------------------------------------------------------- gradients of the dense layer


def product_tile(m, n, k):
    strips = -(-k // 64)
    t256 = rounds(m, n, 256, 256, cus()) * (8 + 1.7 * strips)
    t192 = rounds(m, n, 192, 128, 2 * cus()) * (8 + 1.26 * strips)
    t128 = rounds(m, n, 128, 128, 2 * cus()) * (8 + 1.0 * strips)
    return 256 if t256 <= t192 and t256 <= t128 else 192 if t192 <= t128 else 128


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("tile,rows,cols,depth", [(256, 4088, 3992, 75), (256, 4000, 4088, 136), (192, 6136, 2040, 72), (192, 6100, 2040, 200)])
@pytest.mark.parametrize("which", ["x", "w"])
def test_product_tiles(q, dtype, tile, rows, cols, depth, which):
    """Both gradients in the tiles of 256 x 256 and 192 x 128; sums whose last strip is a part, and rows that end
    inside a tile.  Rows of both operands are whole 16-byte pieces, or other tiles are taken."""
    depth, rows = (-(-depth // 8) * 8, rows) if which == "x" else (depth, -(-rows // 8) * 8)
    assert product_tile(rows, cols, depth) == tile and 2 * tiles(rows, cols, 128, 128) > 2 * cus()
    show("product", which, dtype, tile, rows, cols, depth)
    rng = np.random.default_rng([23, rows, cols, depth])
    a = G.random(rng, (rows, depth) if which == "x" else (depth, rows))
    b = G.random(rng, (depth, cols))
    a64, b64 = G.f64(a), G.f64(b)
    if which == "w":
        a64 = a64.T
    room = torch.full((rows * cols + 16,), 7.0, dtype=dtype, device=DEV)
    out = room[8:8 + rows * cols].view(rows, cols)
    call = q.bf16_gemm_grad_x if which == "x" else q.bf16_gemm_grad_w
    got = call(a, b, out=out, out_dtype=dtype)
    assert bool((room[:8] == 7).all()) and bool((room[8 + rows * cols:] == 7).all()), "writes outside out"
    assert G.close(got, a64 @ b64, (depth + 8) * G.U * (np.abs(a64) @ np.abs(b64)), dtype)
