"""The int4 calls at the ends of their arguments' ranges, against the float64 oracle.

Exact cases as in test_gpu_int4: integer activations in [-4, 4], power-of-two scales and
integer zero points, so every partial result is exact in float32 and the outputs must be
equal bit for bit."""

import numpy as np
import pytest
import torch

from oracle import moe as O
from gpu_util import DEV, show
from test_gpu_int4 import dev, exact_weight, operands, plain64, random_operands, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import weight_quantized_linear_amd as q
    return q


# rows for the streaming form, the tiles that split K and the pipelined ones
@pytest.mark.parametrize("m", [1, 3, 12, 30, 100])
@pytest.mark.parametrize("k", [96, 301])
@pytest.mark.parametrize("group_size", [2 ** 63 - 1, 2 ** 63 - 100, 2 ** 62])
def test_any_group_size_from_k_on_is_one_group(q, m, k, group_size):
    """Through the C entries, whose group size is any int64, and through the binding."""
    rng = np.random.default_rng([30, m, k])
    n, e = 300, 3
    packed, scale, zero = exact_weight(rng, (e,), n, k, k, True)
    x = rng.integers(-4, 5, (m, k)).astype(np.float64)
    w, s, xd, z = operands(packed, scale, zero, x)
    out = torch.full((m, n), 3.0, device=DEV)
    show("int4 group size", m, k, group_size)
    st = q.lib.qlinear_int4_gemm(w[1].data_ptr(), s[1].data_ptr(), z[1].data_ptr(), xd.data_ptr(), out.data_ptr(), q.F32, m,
                                 n, k, group_size, 1.0, None, q._stream(xd))
    assert st == q.OK
    ref, _ = O.int4_linear(packed[1], scale[1], zero[1], x, k)
    assert same(out, ref)
    assert same(q.int4_gemm(w[1], s[1], xd, w_zero=z[1], group_size=2 ** 64 + 32, out_dtype=torch.float32), ref)

    offs, ids = dev(np.array([0, m // 2, m // 2, m], np.int32)), dev(np.array([2, 0, 1], np.int32))
    out.fill_(3.0)
    st = q.lib.qlinear_int4_grouped_gemm(w.data_ptr(), s.data_ptr(), z.data_ptr(), xd.data_ptr(), offs.data_ptr(),
                                         ids.data_ptr(), out.data_ptr(), q.F32, 3, m, e, m, n, k, group_size,
                                         q._stream(xd))
    assert st == q.OK
    ref, _, _ = O.int4_grouped(packed, scale, zero, x, k, offs.cpu().numpy(), ids.cpu().numpy())
    assert same(out, ref)


# rows that end in every 16 rows of a tile, in tiles of several shapes, first and last column tile
@pytest.mark.parametrize("m", [18, 31, 33, 47, 48, 49, 63, 65, 80, 81, 95, 97, 112, 113, 127, 129])
@pytest.mark.parametrize("n", [20001, 33000])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_rows_behind_the_last_one_stay(q, m, n, dt):
    k = 128
    w, s, z, x = random_operands(m + n, m, n, k, 64, True, True)
    rows = 200
    buf = torch.full((m + 2 * rows, n), 7.0, dtype=dt, device=DEV)
    show("int4 rows behind", m, n, dt)
    q.int4_gemm(w, s, x, w_zero=z, group_size=64, out=buf[rows:rows + m], out_dtype=dt)
    assert torch.equal(buf[rows:rows + m], plain64(w, s, z, x, 64).to(dt))
    assert torch.all(buf[:rows] == 7.0) and torch.all(buf[rows + m:] == 7.0)
