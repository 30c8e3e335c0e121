"""GPU parity of the router, the sort, the gather, the combine, the gated
activation and their gradients against the float64 oracle.

Tolerances, with u = 2^-24 (a float32 step is at most u of the value): a sum of
n terms in float32 is off by at most (n + 1) u times the sum of magnitudes; exp,
division and the exponent's subtraction are taken at 16 u together, the
subtraction adding |l - top| u; a bfloat16 output adds half a step, 2^-8."""

import numpy as np
import pytest
import torch

from oracle import moe as O
from gpu_util import DEV, show

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
DTYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module")
def q():
    import weight_quantized_linear_amd as q
    return q


def f64(t):
    return t.double().cpu().numpy()


def random(rng, shape, dtype, std=1.0):
    return torch.from_numpy(rng.normal(size=shape) * std).to(dtype).to(DEV)


def close(out, ref, tau, dtype):
    err = np.abs(f64(out) - ref)
    return bool(np.all(err <= tau + HALF[dtype] * (np.abs(ref) + tau)))


# ---------------------------------------------------------------- router


def check_route(q, logits, top_k, renorm):
    l64 = f64(logits)
    t, e = l64.shape
    ids, w = q.moe_route(logits, top_k, renormalize=renorm)
    rid, rw = O.route(l64, top_k, renorm)
    assert np.array_equal(ids.cpu().numpy(), rid)
    reach = 2 * np.abs(l64).max(1, keepdims=True)
    rel = (e + 16 + reach) * U
    assert np.all(np.abs(f64(w) - rw) <= rel * rw + 2.0 ** -126), "weights"
    rng = np.random.default_rng([5, t, e, top_k])
    dw = random(rng, (t, top_k), torch.float32)
    g = q.moe_route_backward(logits, ids, dw, renormalize=renorm)
    assert g.dtype == logits.dtype
    ref = O.route_backward(l64, rid, f64(dw), renorm)
    full = np.abs(f64(dw)).sum(1, keepdims=True)  # p_e (a_e - mean): both factors off by rel, p_e at most 1
    p = np.ones_like(ref) if renorm else np.exp(l64 - l64.max(1, keepdims=True))
    tau = 2 * rel * p * full + 2.0 ** -126
    assert close(g, ref, tau, logits.dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("t,e,top_k", [(1, 1, 1), (3, 2, 2), (7, 8, 2), (5, 63, 6), (33, 64, 8), (9, 65, 64), (20, 128, 1),
                                       (1000, 60, 4), (4, 129, 8), (40, 256, 8), (3, 257, 10), (6, 512, 22), (5, 1000, 8),
                                       (2, 1024, 64)])
def test_route(q, dtype, renorm, t, e, top_k):
    rng = np.random.default_rng([6, t, e, top_k])
    show("route", dtype, renorm, t, e, top_k)
    check_route(q, random(rng, (t, e), dtype, 2.0), top_k, renorm)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("e", [5, 64, 200])
def test_route_masks_ties_and_extremes(q, dtype, renorm, e):
    rng = np.random.default_rng([7, e])
    low = torch.finfo(dtype).min
    rows = []
    rows.append(np.full(e, -np.inf))                                   # nothing is left
    rows.append(np.where(np.arange(e) == e - 1, 0.5, -np.inf))         # one expert is left
    rows.append(np.where(np.arange(e) < 2, rng.normal(size=e), -np.inf))
    rows.append(np.zeros(e))                                           # all equal
    rows.append(np.where(np.arange(e) % 2 == 0, 0.0, -0.0))            # the two zeros are equal
    rows.append(np.full(e, low))                                       # the lowest value is no mask
    rows.append(np.where(np.arange(e) == 1, low, -np.inf))
    rows.append(np.where(np.arange(e) % 3 == 0, low, rng.normal(size=e)))
    rows.append(np.where(np.arange(e) == 2, 80.0, rng.normal(size=e)))
    rows.append(np.round(rng.normal(size=e)))                          # many ties
    rows.append(np.full(e, -torch.finfo(dtype).max))
    logits = torch.from_numpy(np.stack(rows)).to(dtype).to(DEV)
    show("route extremes", dtype, renorm, e)
    ids, w = q.moe_route(logits, 4, renormalize=renorm)
    rid, rw = O.route(f64(logits), 4, renorm)
    assert np.array_equal(ids.cpu().numpy(), rid)
    assert np.all(np.abs(f64(w) - rw) <= (e + 16 + 200) * U * rw + 2.0 ** -126)
    dw = random(rng, (len(rows), 4), torch.float32)
    g = q.moe_route_backward(logits, ids, dw, renormalize=renorm)
    ref = O.route_backward(f64(logits), rid, f64(dw), renorm)
    full = np.abs(f64(dw)).sum(1, keepdims=True)
    assert np.all(np.abs(f64(g) - ref) <= 2 * (e + 216) * U * full + HALF[dtype] * np.abs(ref) + 2.0 ** -126)
    assert not g[0].any() and not g[1][:e - 1].any()


def test_route_nan_and_infinity(q):
    logits = torch.zeros((3, 6), device=DEV)
    logits[0, 2] = float("nan")
    logits[1, 3] = float("inf")
    logits[2, :] = float("nan")
    show("route nan")
    ids, w = q.moe_route(logits, 2)
    assert ids.cpu().tolist() == [[0, 1], [3, 0], [-1, -1]]
    assert torch.isnan(w).all()


def test_route_backward_ignores_foreign_ids(q):
    logits = torch.randn((2, 8), device=DEV)
    ids = torch.tensor([[1, -1, 99], [-7, 3, 8]], dtype=torch.int32, device=DEV)
    dw = torch.randn((2, 3), device=DEV)
    show("route foreign ids")
    g = q.moe_route_backward(logits, ids, dw, renormalize=False)
    ref = O.route_backward(f64(logits), ids.cpu().numpy(), f64(dw), False)
    assert np.all(np.abs(f64(g) - ref) <= 100 * U * np.abs(f64(dw)).sum(1, keepdims=True))


# ---------------------------------------------------------------- sort


def check_sort(q, ids, e):
    offsets, row_slot, slot_row = q.moe_sort(torch.from_numpy(ids).to(DEV), e)
    ro, rr, rs = O.sort(ids, e)
    assert np.array_equal(offsets.cpu().numpy(), ro)
    assert np.array_equal(row_slot.cpu().numpy(), rr)
    assert np.array_equal(slot_row.cpu().numpy(), rs)


@pytest.mark.parametrize("e", [1, 2, 7, 64, 255, 256, 1024])
@pytest.mark.parametrize("t,top_k", [(1, 1), (8, 8), (63, 1), (65, 1), (512, 8), (513, 8), (4097, 1), (1500, 6), (20000, 10)])
def test_sort(q, e, t, top_k):
    rng = np.random.default_rng([8, e, t, top_k])
    show("sort", e, t, top_k)
    check_sort(q, rng.integers(-1, e, (t, top_k)).astype(np.int32), e)


@pytest.mark.parametrize("t", [100, 9000])
def test_sort_one_sided(q, t):
    """All slots dropped, all on one expert, ids far outside, in descending order."""
    show("sort one-sided", t)
    check_sort(q, np.full((t, 2), -1, np.int32), 5)
    check_sort(q, np.full((t, 2), 4, np.int32), 5)
    check_sort(q, np.where(np.arange(2 * t).reshape(t, 2) % 3 == 0, 2 ** 31 - 1, -2 ** 31).astype(np.int32), 5)
    check_sort(q, (np.arange(2 * t)[::-1].reshape(t, 2) * 1024 // (2 * t)).astype(np.int32), 1024)


def test_sort_large(q):
    rng = np.random.default_rng([9])
    show("sort large")
    check_sort(q, rng.integers(0, 300, (400000, 4)).astype(np.int32), 300)


def test_nothing_to_do(q):
    ids = torch.empty((0, 4), dtype=torch.int32, device=DEV)
    offsets, row_slot, slot_row = q.moe_sort(ids, 6)
    assert offsets.cpu().tolist() == [0] * 7 and row_slot.numel() == 0 and slot_row.shape == (0, 4)
    x = torch.empty((0, 16), device=DEV)
    assert q.moe_gather(x, slot_row).shape == (0, 16) and q.moe_combine(x, slot_row).shape == (0, 16)
    w = torch.empty((0, 4), device=DEV)
    assert q.moe_combine_backward(x, x, slot_row, w)[0].shape == (0, 16)
    assert q.moe_route(x, 4)[0].shape == (0, 4) and q.moe_route_backward(x, ids, w).shape == (0, 16)
    assert q.swiglu(x).shape == (0, 8) and q.swiglu_backward(x[:, :8].contiguous(), x).shape == (0, 16)


# ---------------------------------------------------------------- gather and combine


def slots(rng, t, top_k, dropped):
    ids = rng.integers(0, 5, (t, top_k))
    ids[rng.random((t, top_k)) < dropped] = -1
    return O.sort(ids, 5)[2]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("h", [1, 3, 7, 8, 9, 64, 65, 511, 512, 513, 2048, 4099])
@pytest.mark.parametrize("t,top_k,dropped", [(1, 1, 0.0), (5, 8, 0.3), (70, 3, 0.0), (6, 2, 1.0), (9, 11, 0.1)])
def test_gather_combine_and_gradients(q, dtype, h, t, top_k, dropped):
    rng = np.random.default_rng([20, h, t, top_k])
    place = slots(rng, t, top_k, dropped)
    sr = torch.from_numpy(place.astype(np.int32)).to(DEV)
    x = random(rng, (t, h), dtype)
    show("permute", dtype, h, t, top_k, dropped)
    assert np.array_equal(f64(q.moe_gather(x, sr)), O.gather(f64(x), place))

    rows = random(rng, (t * top_k, h), dtype)
    w = torch.from_numpy(rng.uniform(-1, 1, (t, top_k))).float().to(DEV)
    dead = np.where(place < 0, ~place, -1)
    poisoned = rows.clone()
    poisoned[torch.from_numpy(dead[dead >= 0]).to(DEV)] = float("nan")  # what nothing may read
    wp = torch.where(sr < 0, torch.full_like(w, float("nan")), w)
    for weights, wref in ((wp, f64(w)), (None, None)):
        ref, bound = O.combine(f64(rows), place, wref)
        for out_dtype in DTYPES:
            got = q.moe_combine(poisoned, sr, weights, out_dtype=out_dtype)
            assert close(got, ref, (top_k + 1) * U * bound, out_dtype)

    dy = random(rng, (t, h), dtype)
    gr, gw = q.moe_combine_backward(dy, poisoned, sr, wp)
    rr, rw, bound = O.combine_backward(f64(dy), f64(rows), place, f64(w))
    assert close(gr, rr, U * np.abs(rr), dtype)
    assert np.all(np.abs(f64(gw) - rw) <= (h + 1) * U * bound)


def test_foreign_rows_are_skipped(q):
    """Rows outside 0 .. T * top_k - 1 are neither read nor written."""
    sr = torch.tensor([[0, 7], [-9, 2 ** 31 - 1], [1, -2 ** 31]], dtype=torch.int32, device=DEV)
    x, w = torch.randn((3, 40), device=DEV), torch.ones((3, 2), device=DEV)
    buf = torch.full((8, 40), 5.0, device=DEV)
    show("foreign rows")
    q.moe_gather(x, sr, out=buf[:6])
    assert torch.equal(buf[:2], x[[0, 2]]) and torch.all(buf[2:] == 5.0)
    rows = torch.randn((6, 40), device=DEV)
    out = q.moe_combine(rows, sr, w)
    assert torch.equal(out, torch.stack([rows[0], torch.zeros(40, device=DEV), rows[1]]))
    buf.fill_(5.0)
    _, gw = q.moe_combine_backward(x, rows, sr, w, grad_rows=buf[:6])
    assert torch.equal(buf[:2], x[[0, 2]]) and torch.all(buf[2:] == 5.0)
    assert gw[0, 1] == 0 and not gw[1].any() and gw[2, 1] == 0


def test_rows_beyond_4_gib(q):
    t, top_k, h = 70000, 8, 8192
    ids = torch.randint(0, 16, (t, top_k), device=DEV, dtype=torch.int32)
    _, row_slot, sr = q.moe_sort(ids, 16)
    x = torch.randn((t, h), device=DEV, dtype=torch.float32).bfloat16()
    show("gather beyond 4 GiB")
    xs = q.moe_gather(x, sr)
    for r in (0, 262144, 300001, t * top_k - 1):
        assert torch.equal(xs[r], x[int(row_slot[r]) // top_k])
    back = q.moe_combine(xs, sr)
    assert torch.equal(back, (x.float() * top_k).bfloat16())


@pytest.mark.parametrize("dtype", DTYPES)
def test_calls_larger_than_the_caches(q, dtype):
    """The forms that stream past the caches, against float64 on the device."""
    t, top_k, h = 2700, 6, 4100
    g = torch.Generator(device=DEV).manual_seed(11)
    ids = torch.randint(-1, 40, (t, top_k), generator=g, device=DEV, dtype=torch.int32)
    sr = q.moe_sort(ids, 40)[2]
    x = torch.randn((t, h), generator=g, device=DEV).to(dtype)
    rows = torch.randn((t * top_k, h), generator=g, device=DEV).to(dtype)
    w = torch.rand((t, top_k), generator=g, device=DEV)
    on, place = sr >= 0, torch.where(sr < 0, ~sr, sr).long()
    show("moe large", dtype)
    xs = q.moe_gather(x, sr)
    want = torch.zeros_like(rows)
    want[place[on]] = x.repeat_interleave(top_k, 0).view(t, top_k, h)[on]
    assert torch.equal(xs, want)
    part = rows.double()[place] * torch.where(on, w, 0.0).double()[:, :, None]
    tau = (top_k + 1) * U * part.abs().sum(1)
    ref = part.sum(1)
    assert bool(((q.moe_combine(rows, sr, w).double() - ref).abs() <= tau + HALF[dtype] * (ref.abs() + tau)).all())
    gr, gw = q.moe_combine_backward(x, rows, sr, w)
    ref = torch.zeros_like(rows, dtype=torch.float64)
    ref[place[on]] = (x.double()[:, None, :] * w.double()[:, :, None])[on]
    assert bool(((gr.double() - ref).abs() <= U * ref.abs() + HALF[dtype] * ref.abs() * (1 + U)).all())
    prod = x.double()[:, None, :] * rows.double()[place] * on[:, :, None]
    assert bool(((gw.double() - prod.sum(2)).abs() <= (h + 1) * U * prod.abs().sum(2)).all())


# ---------------------------------------------------------------- gated activation


def test_swiglu_larger_than_the_caches(q):
    m, f = 20000, 1537
    g = torch.Generator(device=DEV).manual_seed(12)
    x = (torch.randn((m, 2 * f), generator=g, device=DEV) * 3).bfloat16()
    dy = torch.randn((m, f), generator=g, device=DEV).bfloat16()
    show("swiglu large")
    gate, up = x.double().split(f, 1)
    sig, rest = torch.sigmoid(gate), torch.sigmoid(-gate)
    ref = gate * sig * up
    tau = 16 * U * ref.abs()
    assert bool(((q.swiglu(x).double() - ref).abs() <= tau + HALF[torch.bfloat16] * (ref.abs() + tau)).all())
    out = q.swiglu_backward(dy, x).double()
    first = dy.double() * up * sig
    for got, ref, size in ((out[:, :f], first * (1 + gate * rest), first.abs() * (1 + gate.abs() * rest)),
                           (out[:, f:], dy.double() * gate * sig, (dy.double() * gate * sig).abs())):
        tau = 16 * U * size
        assert bool(((got - ref).abs() <= tau + HALF[torch.bfloat16] * (ref.abs() + tau)).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,f", [(1, 1), (3, 5), (2, 8), (17, 64), (5, 129), (33, 1536), (300, 77)])
def test_swiglu(q, dtype, m, f):
    rng = np.random.default_rng([21, m, f])
    x = random(rng, (m, 2 * f), dtype, 4.0)
    dy = random(rng, (m, f), dtype)
    show("swiglu", dtype, m, f)
    ref = O.swiglu(f64(x))
    assert close(q.swiglu(x), ref, 16 * U * np.abs(ref), dtype)
    ref, bound = O.swiglu_backward(f64(dy), f64(x))
    assert close(q.swiglu_backward(dy, x), ref, 16 * U * bound, dtype)


def test_swiglu_tails(q):
    """Large gates: neither branch of the sigmoid overflows or cancels."""
    g = torch.tensor([-200.0, -104.0, -88.0, -30.0, -1e-30, 0.0, 1e-30, 30.0, 88.0, 200.0, 3e38], device=DEV)
    x = torch.cat([g, torch.ones_like(g)])[None, :].contiguous()
    dy = torch.ones((1, g.numel()), device=DEV)
    show("swiglu tails")
    ref = O.swiglu(f64(x))
    assert np.all(np.abs(f64(q.swiglu(x)) - ref) <= 16 * U * np.abs(ref) + 2.0 ** -120)
    ref, bound = O.swiglu_backward(f64(dy), f64(x))
    assert np.all(np.abs(f64(q.swiglu_backward(dy, x)) - ref) <= 16 * U * bound + 2.0 ** -120)


# ---------------------------------------------------------------- together


def test_layer_in_a_graph(q):
    """Route, sort, gather, two grouped products, activation, combine and the gradients around them, captured; every
    replay on new inputs equals the eager calls bit for bit."""
    t, e, top_k, h, f = 50, 8, 3, 128, 96
    g = torch.Generator(device=DEV).manual_seed(3)
    w1 = torch.randint(0, 256, (e, 2 * f, h // 2), generator=g, device=DEV, dtype=torch.uint8)
    w2 = torch.randint(0, 256, (e, h, f // 2), generator=g, device=DEV, dtype=torch.uint8)
    s1 = torch.rand((e, 2 * f, h // 32), generator=g, device=DEV).bfloat16() * 0.01
    s2 = torch.rand((e, h, f // 32), generator=g, device=DEV).bfloat16() * 0.01
    x = torch.randn((t, h), generator=g, device=DEV).bfloat16()
    logits = torch.randn((t, e), generator=g, device=DEV)
    dy = torch.randn((t, h), generator=g, device=DEV).bfloat16()
    every = torch.arange(e, dtype=torch.int32, device=DEV)

    def layer():
        ids, w = q.moe_route(logits, top_k)
        offsets, _, sr = q.moe_sort(ids, e)
        xs = q.moe_gather(x, sr)
        up = q.int4_grouped_gemm(w1, s1, xs, offsets, every, group_size=32)
        act = q.swiglu(up)
        rows = q.int4_grouped_gemm(w2, s2, act, offsets, every, group_size=32)
        out = q.moe_combine(rows, sr, w)
        drows, dw = q.moe_combine_backward(dy, rows, sr, w)
        dlogits = q.moe_route_backward(logits, ids, dw)
        dup = q.swiglu_backward(drows[:, :f].contiguous(), up)
        dx = q.moe_combine(dup[:, :h].contiguous(), sr)
        return ids, w, offsets, sr, xs, up, act, rows, out, drows, dw, dlogits, dup, dx

    show("layer: eager")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    show("layer: capture")
    with torch.cuda.graph(graph):
        captured = layer()
    for rep in range(3):
        x.copy_(torch.randn((t, h), generator=g, device=DEV))
        logits.copy_(torch.randn((t, e), generator=g, device=DEV))
        show("layer: replay", rep)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, layer()):
            assert torch.equal(a, b), rep


def test_other_stream(q):
    side = torch.cuda.Stream()
    logits = torch.randn((3000, 64), device=DEV)
    x = torch.randn((3000, 256), device=DEV)
    show("moe on another stream")

    def work():
        ids, w = q.moe_route(logits, 6)
        offsets, row_slot, sr = q.moe_sort(ids, 64)
        return ids, w, offsets, row_slot, sr, q.moe_combine(q.moe_gather(x, sr), sr, w)

    a = work()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = work()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(i, j) for i, j in zip(a, b))
