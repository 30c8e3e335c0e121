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


def equal_or_nan(out, ref):
    """Bit for bit the float64 reference rounded to the output's type; NaN where it is NaN."""
    return torch.equal(torch.nan_to_num(out, nan=0.125, posinf=float("inf"), neginf=float("-inf")),
                       torch.nan_to_num(ref.to(out.dtype), nan=0.125, posinf=float("inf"), neginf=float("-inf")))


def defined64(w, s, z, x, group):
    """x @ D^T elementwise in float64, so that infinities meet exactly the weights of their k."""
    k = x.shape[1]
    codes = torch.stack([w & 15, w >> 4], -1).reshape(w.shape[0], -1)[:, :k].double()
    g = torch.arange(k, device=DEV) // group
    d = (codes - (8.0 if z is None else z.double()[:, g])) * s.double()[:, g]
    return torch.stack([(row[None, :] * d).sum(1) for row in x.double()])


# rows for each form: streaming with K over the waves and not, the tiles that split K, the pipelined ones
FORMS = [(1, 300), (2, 40), (4, 300), (1, 70000), (3, 70000), (9, 300), (12, 9000), (30, 300), (64, 20000), (100, 33000)]


@pytest.mark.parametrize("m,n", FORMS)
@pytest.mark.parametrize("k,group", [(96, 32), (301, 64), (1100, 128), (640, 640)])
def test_infinite_activations_have_the_value_of_the_definition(q, m, n, k, group):
    """inf (code - zero) scale is inf, -inf, or NaN where code = zero; opposite infinities and NaN are NaN; the other rows
    stay exact."""
    w, s, z, x = random_operands(m + n + k, m, n, k, group, k != 301, True)
    inf = float("inf")
    x[0, k // 2] = inf
    if m > 2:
        x[1, 0], x[2, k - 1] = -inf, float("nan")
    if m > 8:
        x[8, 3], x[8, k - 2] = inf, -inf
        x[m - 1, k - 1] = -inf
    show("int4 infinite", m, n, k, group)
    for dt in (torch.float32, torch.bfloat16):
        out = q.int4_gemm(w, s, x, w_zero=z, group_size=group, out_dtype=dt)
        rows = [i for i in (0, 1, 2, 3, 8, m - 1) if i < m]
        assert equal_or_nan(out[rows], defined64(w, s, z, x[rows], group))


@pytest.mark.parametrize("m,n", FORMS)
@pytest.mark.parametrize("k,group", [(96, 32), (301, 64), (1100, 128)])
def test_sums_beyond_float32_in_between(q, m, n, k, group):
    """Activations of up to 2^126 and scales of 2^-23 .. 2^-20: sum x code leaves float32's range, the result does not."""
    w, s, z, x = random_operands(m + n + k + 1, m, n, k, group, True, True)
    x, s = x * 2.0 ** 124, s * 2.0 ** -20
    show("int4 large activations", m, n, k, group)
    ref = plain64(w, s, z, x, group)
    assert bool((x.double().abs().sum(1) * 15 > 3.5e38).all()) and bool((ref.abs() < 3e38).all())
    for dt in (torch.float32, torch.bfloat16):
        assert torch.equal(q.int4_gemm(w, s, x, w_zero=z, group_size=group, out_dtype=dt), ref.to(dt))


@pytest.mark.parametrize("m,n", [(1, 300), (3, 70000), (12, 300), (100, 33000)])
def test_infinite_activations_through_the_epilogue(q, m, n):
    """The residual is the output itself: each of its elements is read before it is written."""
    k, group = 256, 64
    w, s, z, x = random_operands(m + n + 2, m, n, k, group, True, True)
    if m > 1:
        x[0] *= 2.0 ** 124  # sums beyond float32 in between, all partial results exact
    x[m - 1, 7] = float("inf")
    s *= 2.0 ** -20
    bias = torch.randint(-8, 9, (n,), device=DEV).bfloat16()
    out = torch.randint(-8, 9, (m, n), device=DEV).float()
    rows = sorted({0, m // 2, m - 1})
    want = 0.5 * defined64(w, s, z, x[rows], group).float() + bias.float() + out[rows]
    show("int4 infinite epilogue", m, n)
    q.int4_gemm(w, s, x, w_zero=z, group_size=group, out=out, out_dtype=torch.float32, alpha=0.5, bias=bias, residual=out)
    near = torch.isfinite(want)
    assert equal_or_nan(torch.where(near, 0.0, out[rows]), torch.where(near, 0.0, want))
    # three roundings of float32 in 0.5 v + bias + residual, each of values below |v| + 16
    assert bool(((out[rows] - want)[near].abs() <= 4 * 2.0 ** -24 * (want[near].abs() + 32)).all())


@pytest.mark.parametrize("rows,n", [(2, 272), (16, 272), (16, 9000), (70, 272)])
@pytest.mark.parametrize("k,group", [(96, 32), (301, 64), (1100, 128), (640, 640)])
def test_grouped_infinite_and_large_activations(q, rows, n, k, group):
    e, counts = 4, [rows, 0, rows + 1, 1, 2 * rows, rows]
    ids = [3, 0, 1, 2, -1, 0]
    offs = np.concatenate([[0], np.cumsum(counts)])
    t = int(offs[-1])
    w, s, z, x = random_operands(rows + n + k, t, e * n, k, group, True, True)
    w, s, z = w.view(e, n, -1), s.view(e, n, -1) * 2.0 ** -20, z.view(e, n, -1)
    x[::3] *= 2.0 ** 124
    x[1::5, k // 3] = float("inf")
    x[t - 1, k - 1] = float("-inf")
    show("int4 grouped infinite", rows, n, k, group)
    for dt in (torch.float32, torch.bfloat16):
        out = q.int4_grouped_gemm(w, s, x, dev(offs.astype(np.int32)), dev(np.asarray(ids, np.int32)), w_zero=z,
                                  group_size=group, out_dtype=dt)
        for i, (b, c) in enumerate(zip(offs[:-1], offs[1:])):
            if c > b:
                want = defined64(w[ids[i]], s[ids[i]], z[ids[i]], x[b:c], group) if ids[i] >= 0 else \
                    torch.zeros((c - b, n), device=DEV)
                assert equal_or_nan(out[b:c], want)


def test_offsets_that_fall_count_every_row_once(q):
    """Offsets that fall and rise again: 8192 groups would cover all 17 million rows each.  Only the first does; the result of
    the others is undefined, the reads and writes are not."""
    t, groups, e, n, k = 2 ** 24 + 300000, 16384, 3, 4, 2
    w, s, z, x = random_operands(77, 1000, e * n, k, 32, True, True)
    w, s, z = w.view(e, n, -1), s.view(e, n, -1), z.view(e, n, -1)
    x = x.repeat(t // 1000 + 1, 1)[:t].contiguous()
    offs = torch.tensor([0, -1], dtype=torch.int32, device=DEV).repeat(groups // 2 + 1)[:groups + 1].contiguous()
    ids = torch.full((groups,), 1, dtype=torch.int32, device=DEV)
    buf = torch.full((t + 2000, n), 7.0, dtype=torch.bfloat16, device=DEV)
    show("int4 falling offsets", t, groups)
    q.int4_grouped_gemm(w, s, x, offs, ids, w_zero=z, group_size=32, out=buf[1000:1000 + t])
    assert torch.all(buf[:1000] == 7.0) and torch.all(buf[1000 + t:] == 7.0)
    want = plain64(w[1], s[1], z[1], x[:1000], 32).bfloat16()
    assert torch.equal(buf[1000:1000 + t], want.repeat(t // 1000 + 1, 1)[:t])


@pytest.mark.parametrize("t,groups", [(40, 9), (300, 130), (3000, 200), (9000, 70)])
def test_offsets_in_any_order_stay_inside(q, t, groups):
    """Groups that begin behind every earlier end are computed, whatever the other offsets hold; rows behind T stay."""
    rng = np.random.default_rng([31, t, groups])
    e, n, k = 4, 80, 130
    w, s, z, x = random_operands(t + groups, t, e * n, k, 64, True, True)
    w, s, z = w.view(e, n, -1), s.view(e, n, -1), z.view(e, n, -1)
    offs = np.sort(rng.integers(0, t + 1, groups + 1))
    offs[groups // 2] = 2 ** 32 - 1
    offs[[1, groups // 3]] = offs[[groups // 3, 1]]
    ids = rng.integers(-1, e, groups).astype(np.int32)
    buf = torch.full((t + 600, n), 7.0, device=DEV)
    show("int4 offsets in any order", t, groups)
    q.int4_grouped_gemm(w, s, x, dev(offs.astype(np.uint32).view(np.int32)), dev(ids), w_zero=z, group_size=64,
                        out=buf[300:300 + t], out_dtype=torch.float32)
    assert torch.all(buf[:300] == 7.0) and torch.all(buf[300 + t:] == 7.0)
    top, covered = 0, np.zeros(t, int)
    spans = [(min(int(a), t), min(int(b), t)) for a, b in zip(offs[:-1], offs[1:])]
    for b, c in spans:
        covered[b:c] += 1
    for i, (b, c) in enumerate(spans):
        if c > b and b >= top and covered[b:c].max() == 1:
            want = plain64(w[ids[i]], s[ids[i]], z[ids[i]], x[b:c], 64).float() if ids[i] >= 0 else torch.zeros((c - b, n), device=DEV)
            assert torch.equal(buf[300 + b:300 + c], want)
        top = max(top, c)
