"""GPU parity of the int4 linear calls against the float64 oracle.

Exact cases: activations are integers in [-4, 4], scales powers of two, zero
points integers.  A group's sum of x * code and of x then is an integer below
2^24 for K <= 8192, every product with a scale 2^-3 .. 2^0 a multiple of 2^-3,
and all partial results stay below 2^24 * 2^-3 in magnitude at these sizes, so
float32 holds each of them exactly and the result must equal the reference bit
for bit, in any order of summation.

Random cases: with u = 2^-24, a float32 evaluation of the K products, the
groups' corrections and their sum is off by at most (K + 8) u times the bound
the oracle returns; a bfloat16 output adds half a step, 2^-8 of the value."""

import numpy as np
import pytest
import torch

from oracle import moe as O
from gpu_util import DEV, show

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module")
def q():
    import weight_quantized_linear_amd as q
    return q


def exact_weight(rng, lead, n, k, group, zeros):
    groups = -(-k // group)
    packed = rng.integers(0, 256, (*lead, n, (k + 1) // 2), dtype=np.uint8)
    scale = 2.0 ** rng.integers(-3, 1, (*lead, n, groups))
    zero = rng.integers(0, 16, (*lead, n, groups)).astype(np.uint8) if zeros else None
    return packed, scale, zero


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def operands(packed, scale, zero, x):
    return dev(packed), dev(scale, torch.bfloat16), dev(x, torch.bfloat16), None if zero is None else dev(zero)


def same(out, ref):
    """Bit for bit the reference rounded to the output's type."""
    return torch.equal(out.cpu(), torch.from_numpy(ref).to(out.dtype))


# every row count up to 4 and the edges of the row tiles; K around the chunk (32), the strip (128) and their odd ends
@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 16, 17, 32, 33, 64, 65, 130, 200])
@pytest.mark.parametrize("k,group", [(1, 32), (31, 32), (33, 32), (64, 32), (96, 64), (127, 128), (128, 128), (129, 64),
                                     (257, 32), (640, 128), (1000, 256), (2050, 64), (300, 300), (2048, 4096)])
def test_exact(q, m, k, group):
    rng = np.random.default_rng([10, m, k, group])
    for n, zeros, dt in ((70, True, torch.float32), (257, False, torch.bfloat16)):
        show("int4 exact", m, n, k, group, zeros)
        packed, scale, zero = exact_weight(rng, (), n, k, group, zeros)
        x = rng.integers(-4, 5, (m, k)).astype(np.float64)
        ref, _ = O.int4_linear(packed, scale, zero, x, group)
        w, s, xd, z = operands(packed, scale, zero, x)
        assert same(q.int4_gemm(w, s, xd, w_zero=z, group_size=group, out_dtype=dt), ref)


@pytest.mark.parametrize("m", [1, 2, 7, 48, 100])
@pytest.mark.parametrize("n,k", [(1, 128), (15, 256), (4096, 512), (9000, 160), (20000, 96)])
def test_exact_wide(q, m, n, k):
    rng = np.random.default_rng([11, m, n, k])
    show("int4 exact wide", m, n, k)
    packed, scale, zero = exact_weight(rng, (), n, k, 32, True)
    x = rng.integers(-4, 5, (m, k)).astype(np.float64)
    ref, _ = O.int4_linear(packed, scale, zero, x, 32)
    w, s, xd, z = operands(packed, scale, zero, x)
    assert same(q.int4_gemm(w, s, xd, w_zero=z, group_size=32, out_dtype=torch.float32), ref)


@pytest.mark.parametrize("m", [1, 9, 70])
def test_every_code_and_zero_point(q, m):
    """One-hot activations read the dequantised weight back: all 16 codes in all 8 places of a dword, zero points 0 .. 255."""
    n, k = 256, 128
    codes = (np.arange(n)[:, None] + np.arange(k)[None, :] * 5) % 16
    packed = (codes[:, 0::2] | codes[:, 1::2] << 4).astype(np.uint8)
    zero = np.arange(n, dtype=np.uint8)[:, None].repeat(4, 1)
    scale = np.ones((n, 4))
    for k0 in range(0, k, m):
        x = np.zeros((m, k))
        for i in range(m):
            x[i, (k0 + i) % k] = 1.0
        show("int4 codes", m, k0)
        w, s, xd, z = operands(packed, scale, zero, x)
        out = q.int4_gemm(w, s, xd, w_zero=z, group_size=32, out_dtype=torch.float32)
        assert same(out, x @ (codes - zero[:, :1].astype(np.float64)).T)


@pytest.mark.parametrize("m,n,k,group", [(1, 4096, 4096, 128), (2, 1000, 14336, 64), (4, 512, 8190, 32), (16, 2048, 4096, 128),
                                         (40, 1024, 2048, 64), (150, 700, 3000, 128)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_random(q, m, n, k, group, dt):
    rng = np.random.default_rng([12, m, n, k])
    groups = -(-k // group)
    packed = rng.integers(0, 256, (n, (k + 1) // 2), dtype=np.uint8)
    scale = dev(rng.uniform(0.5, 1.5, (n, groups)) * 0.01).to(torch.bfloat16)
    zero = rng.integers(0, 16, (n, groups)).astype(np.uint8)
    x = dev(rng.normal(size=(m, k))).to(torch.bfloat16)
    show("int4 random", m, n, k, group, dt)
    out = q.int4_gemm(dev(packed), scale, x, w_zero=dev(zero), group_size=group, out_dtype=dt)
    ref, bound = O.int4_linear(packed, scale.double().cpu().numpy(), zero, x.double().cpu().numpy(), group)
    tau = (k + 8) * U * bound
    err = np.abs(out.double().cpu().numpy() - ref)
    assert np.all(err <= tau + HALF[dt] * (np.abs(ref) + tau)), float((err / bound).max())


@pytest.mark.parametrize("m", [1, 6, 80])
@pytest.mark.parametrize("k", [64, 127, 250])
def test_views_off_alignment_and_writes_inside_out(q, m, k):
    """Weights, zero points and activations that start off every boundary, inside buffers whose other bytes are extreme
    (codes 15, NaN activations, NaN scales); nothing outside ``out`` changes."""
    rng = np.random.default_rng([13, m, k])
    n, group = 37, 64
    packed, scale, zero = exact_weight(rng, (), n, k, group, True)
    x = rng.integers(-4, 5, (m, k)).astype(np.float64)
    ref, _ = O.int4_linear(packed, scale, zero, x, group)

    def inside(t, shift, fill):
        flat = torch.full((t.numel() + 64,), fill, dtype=t.dtype, device=DEV)
        flat[shift:shift + t.numel()] = t.reshape(-1)
        return flat[shift:shift + t.numel()].view(t.shape)

    w, s, xd, z = operands(packed, scale, zero, x)
    for shift in (1, 3, 7):
        show("int4 views", m, k, shift)
        buf = torch.full((m * n + 32,), 7.0, dtype=torch.float32, device=DEV)
        out = buf[shift:shift + m * n].view(m, n)
        q.int4_gemm(inside(w, shift, 255), inside(s, shift, float("nan")), inside(xd, shift, float("nan")),
                    w_zero=inside(z, shift, 255), group_size=group, out=out, out_dtype=torch.float32)
        assert same(out, ref)
        assert torch.all(buf[:shift] == 7.0) and torch.all(buf[shift + m * n:] == 7.0)


@pytest.mark.parametrize("m", [1, 2, 12, 90])
def test_nan_scale_and_nonfinite_rows_stay_in_their_place(q, m):
    rng = np.random.default_rng([14, m])
    n, k, group = 100, 300, 64
    packed, scale, zero = exact_weight(rng, (), n, k, group, True)
    x = rng.integers(-4, 5, (m, k)).astype(np.float64)
    ref, _ = O.int4_linear(packed, scale, zero, x, group)
    w, s, xd, z = operands(packed, scale, zero, x)
    s[41, 4] = float("nan")
    if m > 1:
        xd[m - 1, 77] = float("inf")
    show("int4 nan", m)
    out = q.int4_gemm(w, s, xd, w_zero=z, group_size=group, out_dtype=torch.float32).cpu().numpy()
    rows = slice(0, m - 1 if m > 1 else 1)
    cols = np.arange(n) != 41
    assert np.isnan(out[:, 41]).all()
    assert np.array_equal(out[rows][:, cols], ref[rows][:, cols].astype(np.float32))
    if m > 1:
        assert not np.isfinite(out[m - 1]).any()


@pytest.mark.parametrize("m", [1, 3, 20, 70])
def test_epilogue(q, m):
    """Power-of-two row and column scales, integer bias and residual, ReLU: exact."""
    rng = np.random.default_rng([15, m])
    n, k = 130, 256
    packed, scale, zero = exact_weight(rng, (), n, k, 128, True)
    x = rng.integers(-4, 5, (m, k)).astype(np.float64)
    ref, _ = O.int4_linear(packed, scale, zero, x, 128)
    rs, cs = 2.0 ** rng.integers(-1, 2, m), 2.0 ** rng.integers(-1, 2, n)
    bias, res = rng.integers(-8, 9, n).astype(np.float64), rng.integers(-8, 9, (m, n)).astype(np.float64)
    want = np.maximum(0.5 * ref * rs[:, None] * cs[None, :] + bias, 0.0) + res
    w, s, xd, z = operands(packed, scale, zero, x)
    show("int4 epilogue", m)
    out = q.int4_gemm(w, s, xd, w_zero=z, group_size=128, out_dtype=torch.float32, alpha=0.5, row_scale=dev(rs, torch.float32),
                      col_scale=dev(cs, torch.float32), bias=dev(bias, torch.bfloat16), residual=dev(res, torch.float32),
                      activation="relu")
    assert same(out, want)


@pytest.mark.parametrize("m", [1, 5, 65])
def test_weight_beyond_4_gib(q, m):
    """The last rows of a weight whose byte offsets pass 2^32."""
    n, k, group = 70000, 131072, 128
    rng = np.random.default_rng([16, m])
    w = torch.zeros((n, k // 2), dtype=torch.uint8, device=DEV)
    s = torch.ones((n, k // group), dtype=torch.bfloat16, device=DEV)
    z = torch.zeros((n, k // group), dtype=torch.uint8, device=DEV)
    tail = rng.integers(0, 256, (3, 64), dtype=np.uint8)
    w[-3:, -64:] = dev(tail)
    x = torch.zeros((m, k), dtype=torch.bfloat16, device=DEV)
    xt = rng.integers(-4, 5, (m, 128)).astype(np.float64)
    x[:, -128:] = dev(xt, torch.bfloat16)
    show("int4 beyond 4 GiB", m)
    out = q.int4_gemm(w, s, x, w_zero=z, group_size=group, out_dtype=torch.float32)
    ref, _ = O.int4_linear(tail, np.ones((3, 1)), np.zeros((3, 1)), xt, 128)
    assert same(out[:, -3:], ref)
    assert not out[:, :-3].any()


def plain64(packed, scale, zero, x, group):
    """x @ D^T by the definition in float64 torch on the device: for sizes the numpy oracle is slow at."""
    k = x.shape[1]
    codes = torch.stack([packed & 15, packed >> 4], -1).reshape(packed.shape[0], -1)[:, :k].double()
    g = torch.arange(k, device=DEV) // group
    z = 8.0 if zero is None else zero.double()[:, g]
    return x.double() @ ((codes - z) * scale.double()[:, g]).t().contiguous()


def random_operands(seed, m, n, k, group, zeros, exact):
    g = torch.Generator(device=DEV).manual_seed(seed)
    groups = -(-k // group)
    w = torch.randint(0, 256, (n, (k + 1) // 2), generator=g, device=DEV, dtype=torch.uint8)
    z = torch.randint(0, 16, (n, groups), generator=g, device=DEV, dtype=torch.uint8) if zeros else None
    if exact:
        s = torch.exp2(torch.randint(-3, 1, (n, groups), generator=g, device=DEV).float()).bfloat16()
        x = torch.randint(-4, 5, (m, k), generator=g, device=DEV).bfloat16()
    else:
        s = (torch.rand((n, groups), generator=g, device=DEV) * 0.01 + 0.005).bfloat16()
        x = torch.randn((m, k), generator=g, device=DEV).bfloat16()
    return w, s, z, x


# sizes for the tiles of 32x32, 64x128, 128x256, 128x128, 32x128 and 64x256; K of one strip, of a few and of many,
# whole and partial, so that every phase of the pipeline and every number of filled correction slots comes up
@pytest.mark.parametrize("m,n", [(20, 33000), (40, 20000), (100, 33000), (100, 20001), (250, 4096), (40, 40000)])
@pytest.mark.parametrize("k,group", [(96, 32), (128, 128), (129, 64), (256, 32), (385, 128), (640, 64), (1000, 32), (1152, 128),
                                     (2050, 256), (1023, 64), (700, 700)])
def test_exact_big_tiles(q, m, n, k, group):
    for zeros, dt in ((True, torch.float32), (False, torch.bfloat16)):
        show("int4 big tiles", m, n, k, group, zeros)
        w, s, z, x = random_operands(m * n + k, m, n, k, group, zeros, True)
        out = q.int4_gemm(w, s, x, w_zero=z, group_size=group, out_dtype=dt)
        assert torch.equal(out, plain64(w, s, z, x, group).to(dt))


@pytest.mark.parametrize("m,n,k,group", [(24, 33000, 1536, 128), (300, 20000, 1500, 64), (128, 33100, 640, 32)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_random_big_tiles(q, m, n, k, group, dt):
    w, s, z, x = random_operands(m + n, m, n, k, group, True, False)
    show("int4 random big tiles", m, n, k, group, dt)
    out = q.int4_gemm(w, s, x, w_zero=z, group_size=group, out_dtype=dt).double()
    ref = plain64(w, s, z, x, group)
    size = plain64(w, s, torch.zeros_like(z), x.abs(), group) + plain64(torch.zeros_like(w), s, z, x.abs(), group).abs()
    tau = (k + 8) * U * size
    assert bool(((out - ref).abs() <= tau + HALF[dt] * (ref.abs() + tau)).all())


@pytest.mark.parametrize("m,n", [(20, 33000), (40, 20000), (100, 33000), (70, 20001)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_big_tiles_write_inside_out_and_take_the_epilogue(q, m, n, dt):
    k = 256
    w, s, z, x = random_operands(n, m, n, k, 64, True, True)
    ref = plain64(w, s, z, x, 64)
    buf = torch.full((m * n + 4096,), 7.0, dtype=dt, device=DEV)
    show("int4 big tiles bounds", m, n, dt)
    q.int4_gemm(w, s, x, w_zero=z, group_size=64, out=buf[2048:2048 + m * n].view(m, n), out_dtype=dt)
    assert torch.equal(buf[2048:2048 + m * n].view(m, n), ref.to(dt))
    assert torch.all(buf[:2048] == 7.0) and torch.all(buf[2048 + m * n:] == 7.0)
    bias = torch.randint(-8, 9, (n,), device=DEV).bfloat16()
    res = torch.randint(-8, 9, (m, n), device=DEV).float()
    out = q.int4_gemm(w, s, x, w_zero=z, group_size=64, out_dtype=dt, alpha=0.5, bias=bias, residual=res, activation="relu")
    assert torch.equal(out, (torch.relu(0.5 * ref + bias.double()) + res.double()).to(dt))


def test_big_tile_keeps_nonfinite_values_in_their_place(q):
    """A NaN scale stays in its column; infinities and NaN of x in their rows, also where the row's group follows others."""
    m, n, k = 100, 33000, 512
    w, s, z, x = random_operands(5, m, n, k, 64, True, True)
    ref = plain64(w, s, z, x, 64).float()
    s[777, 3] = float("nan")
    x[5, 70], x[63, 200], x[99, 511] = float("inf"), float("nan"), float("-inf")
    show("int4 big tiles non-finite")
    out = q.int4_gemm(w, s, x, w_zero=z, group_size=64, out_dtype=torch.float32)
    rows = torch.ones(m, dtype=torch.bool, device=DEV)
    rows[[5, 63, 99]] = False
    cols = torch.ones(n, dtype=torch.bool, device=DEV)
    cols[777] = False
    assert torch.equal(out[rows][:, cols], ref[rows][:, cols])
    assert torch.isnan(out[:, 777]).all() and not torch.isfinite(out[~rows]).any()


def test_no_rows(q):
    w, s = torch.zeros((8, 32), dtype=torch.uint8, device=DEV), torch.ones((8, 2), dtype=torch.bfloat16, device=DEV)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    assert q.int4_gemm(w, s, x, group_size=32).shape == (0, 8)


def test_binding_checks_shapes(q):
    w, s = torch.zeros((8, 32), dtype=torch.uint8, device=DEV), torch.ones((8, 2), dtype=torch.bfloat16, device=DEV)
    x = torch.zeros((2, 64), dtype=torch.bfloat16, device=DEV)
    z = torch.zeros((8, 2), dtype=torch.uint8, device=DEV)
    q.int4_gemm(w, s, x, w_zero=z, group_size=32)
    for kw in (dict(group_size=64), dict(group_size=16), dict(group_size=0), dict(group_size=32, w_zero=z[:4]),
               dict(group_size=32, w_zero=z.int())):
        with pytest.raises(ValueError):
            q.int4_gemm(w, s, x, **kw)
    with pytest.raises(ValueError):
        q.int4_gemm(w, s, x[:, :62], group_size=32)
    with pytest.raises(TypeError):
        q.int4_gemm(w, s, x.float(), group_size=32)


# ---------------------------------------------------------------- grouped

GROUPS = [
    ([0, 1, 1, 4, 10], [2, 0, -1, 1]),                    # an empty group, one switched off, short ones
    ([0, 0, 150, 150, 290], [1, 3, 0, 9]),                # long groups, an id beyond the experts
    ([3, 20, 37, 37, 60], [0, 3, 2, 1]),                  # rows in front of the first group stay
    ([0, 5, 400, 4000000000, 4294967295], [3, 2, 1, 0]),  # offsets past T are clipped
]


@pytest.mark.parametrize("case", range(len(GROUPS)))
@pytest.mark.parametrize("n,k,group,t", [(70, 128, 32, 300), (300, 200, 64, 300), (64, 71, 128, 300), (130, 512, 128, 20)])
def test_grouped_exact(q, case, n, k, group, t):
    rng = np.random.default_rng([17, case, n, k])
    offs, ids = GROUPS[case]
    packed, scale, zero = exact_weight(rng, (4,), n, k, group, case % 2 == 0)
    x = rng.integers(-4, 5, (t, k)).astype(np.float64)
    ref, _, written = O.int4_grouped(packed, scale, zero, x, group, offs, ids)
    w, s, xd, z = operands(packed, scale, zero, x)
    offs_d = torch.from_numpy(np.asarray(offs, np.uint32).view(np.int32)).to(DEV)
    for dt in (torch.float32, torch.bfloat16):
        for most in (0, t):
            show("int4 grouped", case, n, k, group, t, dt, most)
            out = torch.full((t, n), 3.0, dtype=dt, device=DEV)
            q.int4_grouped_gemm(w, s, xd, offs_d, dev(np.asarray(ids, np.int32)), w_zero=z, group_size=group, out=out,
                                out_dtype=dt, max_tokens_per_group=most)
            assert same(out[torch.from_numpy(written).to(DEV)], ref[written])
            assert torch.all(out[torch.from_numpy(~written).to(DEV)] == 3.0)


@pytest.mark.parametrize("groups,t", [(1, 1), (1, 700), (65, 65), (130, 40), (200, 3000), (1000, 500)])
def test_grouped_many_groups(q, groups, t):
    rng = np.random.default_rng([18, groups, t])
    e, n, k = 7, 48, 160
    packed, scale, zero = exact_weight(rng, (e,), n, k, 32, True)
    offs = np.concatenate([[0], np.sort(rng.integers(0, t + 1, groups - 1)), [t]])
    ids = rng.integers(-1, e, groups).astype(np.int32)
    x = rng.integers(-4, 5, (t, k)).astype(np.float64)
    ref, _, written = O.int4_grouped(packed, scale, zero, x, 32, offs, ids)
    w, s, xd, z = operands(packed, scale, zero, x)
    show("int4 grouped many", groups, t)
    out = q.int4_grouped_gemm(w, s, xd, dev(offs.astype(np.int32)), dev(ids), w_zero=z, group_size=32, out_dtype=torch.float32)
    assert written.all() and same(out, ref)


# one to six rows a group, about 16 in few columns and in many, over 32: each form of the walk; K long, odd and short
@pytest.mark.parametrize("rows,n", [(1, 272), (3, 272), (16, 272), (16, 9000), (70, 272), (300, 272)])
@pytest.mark.parametrize("k,group", [(1100, 32), (1024, 64), (897, 128), (2000, 512), (33, 32)])
def test_grouped_forms(q, rows, n, k, group):
    e, groups = 5, 7
    rng = np.random.default_rng([23, rows, k])
    counts = rng.integers(0, 2 * rows + 1, groups)
    counts[0], counts[3] = rows, 0
    offs = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).to(DEV)
    ids = torch.tensor([4, 0, -1, 2, 1, 3, 4], dtype=torch.int32, device=DEV)
    t = int(counts.sum())
    w, s, z, x = random_operands(rows + k, t, e * n, k, group, True, True)
    w, s, z = w.view(e, n, -1), s.view(e, n, -1), z.view(e, n, -1)
    for dt in (torch.float32, torch.bfloat16):
        show("int4 grouped forms", rows, k, group, dt)
        out = torch.full((t + 2, n), 3.0, dtype=dt, device=DEV)
        q.int4_grouped_gemm(w, s, x, offs, ids, w_zero=z, group_size=group, out=out[:t], out_dtype=dt)
        assert torch.all(out[t:] == 3.0)
        for i, (b, c) in enumerate(zip(offs[:-1].tolist(), offs[1:].tolist())):
            x_i, e_i = x[b:c], int(ids[i])
            want = plain64(w[e_i], s[e_i], z[e_i], x_i, group) if e_i >= 0 else torch.zeros((c - b, n), device=DEV)
            assert torch.equal(out[b:c], want.to(dt))


def test_grouped_more_groups_than_a_block_counts(q):
    """Most of 40000 groups are empty; the rows' groups lie before and behind each launch's last group."""
    groups, e, n, k = 40000, 3, 48, 64
    at = [0, 1, 16383, 16384, 20000, 32767, 32768, 39999]
    counts = torch.zeros(groups, dtype=torch.int64)
    counts[at] = torch.tensor([2, 1, 5, 1, 3, 4, 1, 2])
    offs = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
    ids = torch.arange(groups) % e
    w, s, z, x = random_operands(9, int(counts.sum()), e * n, k, 32, True, True)
    w, s, z = w.view(e, n, -1), s.view(e, n, -1), z.view(e, n, -1)
    show("int4 grouped 40000")
    out = q.int4_grouped_gemm(w, s, x, offs.int().to(DEV), ids.int().to(DEV), w_zero=z, group_size=32, out_dtype=torch.float32)
    for i in at:
        b, c = int(offs[i]), int(offs[i + 1])
        assert torch.equal(out[b:c], plain64(w[i % e], s[i % e], z[i % e], x[b:c], 32).float())


def test_other_stream_and_same_bits_again(q):
    rng = np.random.default_rng([19])
    packed, scale, zero = exact_weight(rng, (), 512, 1024, 128, True)
    w, s, _, z = operands(packed, scale, zero, np.zeros((1, 1024)))
    side = torch.cuda.Stream()
    for m in (1, 12, 100):
        x = torch.randn((m, 1024), device=DEV).bfloat16()
        show("int4 stream", m)
        a = q.int4_gemm(w, s, x, w_zero=z, out_dtype=torch.float32)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            b = q.int4_gemm(w, s, x, w_zero=z, out_dtype=torch.float32)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(a, b)
