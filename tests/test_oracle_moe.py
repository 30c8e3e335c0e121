"""The float64 oracle of the MoE operators against other statements of the
same definitions: element-by-element loops, differences for the gradients,
torch's softmax; and the refusals of the calls (no device needed)."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import moe as O


@pytest.fixture(scope="module")
def q():
    import weight_quantized_linear_amd as q
    return q


@pytest.mark.parametrize("k,group,with_zero", [(7, 32, True), (64, 32, False), (71, 32, True), (130, 64, True), (5, 5, False)])
def test_int4_linear_by_elements(k, group, with_zero):
    rng = np.random.default_rng([1, k, group])
    n, m, groups = 3, 2, -(-k // group)
    packed = rng.integers(0, 256, (n, (k + 1) // 2), dtype=np.uint8)
    scale = rng.normal(size=(n, groups))
    zero = rng.integers(0, 16, (n, groups)) if with_zero else None
    x = rng.normal(size=(m, k))
    out, _ = O.int4_linear(packed, scale, zero, x, group)
    for i in range(m):
        for j in range(n):
            total = 0.0
            for c in range(k):
                byte = int(packed[j, c // 2])
                code = byte // 16 if c % 2 else byte % 16
                z = 8 if zero is None else int(zero[j, c // group])
                total += x[i, c] * (code - z) * scale[j, c // group]
            assert abs(out[i, j] - total) <= 1e-12 * (1 + abs(total))


def test_route_against_softmax_and_masks():
    rng = np.random.default_rng(2)
    logits = rng.normal(size=(20, 9))
    ids, w = O.route(logits, 9, False)
    assert np.allclose(np.take_along_axis(torch.softmax(torch.from_numpy(logits), 1).numpy(), ids.astype(int), 1), w)
    ids, w = O.route(logits, 3, True)
    assert np.allclose(w.sum(1), 1.0) and np.all(np.diff(w, axis=1) <= 0)
    logits[0, :] = -np.inf
    logits[1, 2:] = -np.inf
    logits[2, :] = 1.5
    ids, w = O.route(logits, 3, True)
    assert ids[0].tolist() == [-1, -1, -1] and w[0].tolist() == [0, 0, 0]
    assert sorted(ids[1][:2].tolist()) == [0, 1] and ids[1][2] == -1 and w[1][2] == 0
    assert ids[2].tolist() == [0, 1, 2] and np.allclose(w[2], 1 / 3)


@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_against_differences(renorm):
    rng = np.random.default_rng(3)
    logits = rng.normal(size=(4, 8))
    logits[1, 5:] = -np.inf
    ids, _ = O.route(logits, 3, renorm)
    dw = rng.normal(size=(4, 3))
    grad = O.route_backward(logits, ids, dw, renorm)

    def loss(a):
        total = 0.0
        for i in range(4):
            pool = a[i][ids[i]] if renorm else a[i]
            total += (dw[i] * np.exp(a[i][ids[i]]) / np.exp(pool).sum()).sum()
        return total

    h = 1e-5
    for i in range(4):
        for e in range(8):
            if logits[i, e] == -np.inf:
                assert grad[i, e] == 0.0
                continue
            up, down = logits.copy(), logits.copy()
            up[i, e] += h
            down[i, e] -= h
            assert abs((loss(up) - loss(down)) / (2 * h) - grad[i, e]) < 1e-8


def test_sort_gather_combine_and_gradients():
    rng = np.random.default_rng(4)
    t, k, e, h = 6, 3, 4, 5
    ids = rng.integers(-1, e + 1, (t, k))
    offsets, row_slot, slot_row = O.sort(ids, e)
    assert offsets[0] == 0 and offsets[-1] == ((ids >= 0) & (ids < e)).sum()
    for ex in range(e):  # the rows of an expert are its slots, ascending
        assert row_slot[offsets[ex]:offsets[ex + 1]].tolist() == np.flatnonzero(ids.reshape(-1) == ex).tolist()
    assert np.all(row_slot[offsets[-1]:] < 0)
    back = np.where(slot_row < 0, ~slot_row, slot_row).reshape(-1)
    assert sorted(back.tolist()) == list(range(t * k))
    x, w = rng.normal(size=(t, h)), rng.normal(size=(t, k))
    xs = O.gather(x, slot_row)
    live = (ids >= 0) & (ids < e)
    assert np.allclose(O.combine(xs, slot_row, w)[0], x * np.where(live, w, 0).sum(1)[:, None])
    rows, dy, drows = rng.normal(size=(t * k, h)), rng.normal(size=(t, h)), rng.normal(size=(t * k, h))
    gr, gw, _ = O.combine_backward(dy, rows, slot_row, w)
    d, dwt = rng.normal(size=rows.shape), rng.normal(size=w.shape)
    eps = 1e-6
    diff = ((O.combine(rows + eps * d, slot_row, w + eps * dwt)[0]
             - O.combine(rows - eps * d, slot_row, w - eps * dwt)[0]) * dy).sum() / (2 * eps)
    assert abs(diff - (gr * d).sum() - (gw * dwt).sum()) < 1e-7
    # the gradient of gather is combine without weights: <gather(x), d> = <x, combine(d)>
    assert np.isclose((xs * drows).sum(), (x * O.combine(drows, slot_row, None)[0]).sum())


def test_swiglu_backward_against_differences():
    rng = np.random.default_rng(5)
    x, dy, d = rng.normal(size=(3, 8)) * 3, rng.normal(size=(3, 4)), rng.normal(size=(3, 8))
    g, _ = O.swiglu_backward(dy, x)
    eps = 1e-6
    assert abs(((O.swiglu(x + eps * d) - O.swiglu(x - eps * d)) * dy).sum() / (2 * eps) - (g * d).sum()) < 1e-7
    assert np.allclose(O.swiglu(x), torch.nn.functional.silu(torch.from_numpy(x[:, :4])).numpy() * x[:, 4:])


FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p(0x10001)


def test_int4_refusals(q):
    ok = [FAKE, FAKE, None, FAKE, FAKE, 0, 4, 8, 64, 32, 1.0, None, None]
    for i, bad in [(0, None), (1, None), (3, None), (4, None), (5, 2), (5, 9), (6, -1), (7, 0), (8, 0), (8, -3), (9, 16),
                   (9, 0), (9, -32), (9, 48), (1, ODD), (3, ODD), (4, ODD), (7, 1 << 62)]:
        a = list(ok)
        a[i] = bad
        assert q.lib.qlinear_int4_gemm(*a) == q.ERR_INVALID_ARG, (i, bad)
    ok = [FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, 0, 2, 4, 3, 4, 8, 64, 32, None]
    for i, bad in [(0, None), (1, None), (3, None), (4, None), (5, None), (6, None), (7, 2), (8, 0), (8, 65536), (9, -1),
                   (10, 0), (11, -1), (11, 1 << 31), (12, 0), (13, 0), (14, 33), (4, ODD), (5, ODD), (6, ODD)]:
        a = list(ok)
        a[i] = bad
        assert q.lib.qlinear_int4_grouped_gemm(*a) == q.ERR_INVALID_ARG, (i, bad)


def test_int4_refuses_a_k_of_2_to_23(q):
    a = [FAKE, FAKE, None, FAKE, FAKE, 0, 4, 8, 1 << 23, 1 << 23, 1.0, None, None]
    assert q.lib.qlinear_int4_gemm(*a) == q.ERR_INVALID_ARG
    a = [FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, 0, 2, 4, 3, 4, 8, 1 << 23, 32, None]
    assert q.lib.qlinear_int4_grouped_gemm(*a) == q.ERR_INVALID_ARG


def test_moe_refusals(q):
    L, bad_arg = q.lib, q.ERR_INVALID_ARG

    def all_refused(fn, ok, bads):
        for i, bad in bads:
            a = list(ok)
            a[i] = bad
            assert fn(*a) == bad_arg, (fn, i, bad)

    all_refused(L.qlinear_moe_route, [FAKE, 0, FAKE, FAKE, 4, 8, 2, 1, None],
                [(0, None), (2, None), (3, None), (1, 2), (4, -1), (4, 1 << 31), (5, 0), (5, 1025), (6, 0), (6, 9), (0, ODD),
                 (2, ODD), (3, ODD)])
    all_refused(L.qlinear_moe_route, [FAKE, 0, FAKE, FAKE, 4, 100, 2, 1, None], [(6, 65)])
    all_refused(L.qlinear_moe_route_backward, [FAKE, 0, FAKE, FAKE, FAKE, 4, 8, 2, 1, None],
                [(0, None), (2, None), (3, None), (4, None), (1, 7), (5, -1), (6, 0), (7, 9), (4, ODD)])
    all_refused(L.qlinear_moe_sort, [FAKE, FAKE, FAKE, FAKE, 8, 4, None, 0, None],
                [(0, None), (1, None), (2, None), (3, None), (4, -1), (4, 1 << 31), (5, 0), (5, 1025), (7, 16), (7, -1),
                 (0, ODD), (1, ODD), (2, ODD), (3, ODD)])
    need = ctypes.c_int64(0)
    assert L.qlinear_moe_sort_workspace_size(1 << 20, 64, ctypes.byref(need)) == q.OK and need.value > 0
    assert L.qlinear_moe_sort(FAKE, FAKE, FAKE, FAKE, 1 << 20, 64, FAKE, need.value - 1, None) == bad_arg
    assert L.qlinear_moe_sort(FAKE, FAKE, FAKE, FAKE, 1 << 20, 64, ctypes.c_void_p(0x10004), need.value, None) == bad_arg
    assert L.qlinear_moe_sort_workspace_size(8, 4, None) == bad_arg
    assert L.qlinear_moe_sort_workspace_size(-1, 4, ctypes.byref(need)) == bad_arg
    all_refused(L.qlinear_moe_gather, [FAKE, FAKE, FAKE, 0, 4, 2, 8, None],
                [(0, None), (1, None), (2, None), (3, 2), (4, -1), (4, 1 << 31), (5, 0), (5, 65), (6, 0), (0, ODD), (2, ODD)])
    all_refused(L.qlinear_moe_combine, [FAKE, 0, FAKE, FAKE, FAKE, 0, 4, 2, 8, None],
                [(0, None), (2, None), (4, None), (1, 2), (5, 3), (6, -1), (7, 0), (8, 0), (0, ODD), (3, ODD), (4, ODD)])
    all_refused(L.qlinear_moe_combine_backward, [FAKE, FAKE, 0, FAKE, FAKE, FAKE, FAKE, 4, 2, 8, None],
                [(0, None), (1, None), (3, None), (4, None), (5, None), (6, None), (2, 2), (7, -1), (8, 65), (9, 0), (5, ODD)])
    all_refused(L.qlinear_swiglu, [FAKE, FAKE, 0, 4, 8, None], [(0, None), (1, None), (2, 2), (3, -1), (4, 0), (0, ODD)])
    all_refused(L.qlinear_swiglu_backward, [FAKE, FAKE, FAKE, 0, 4, 8, None],
                [(0, None), (1, None), (2, None), (3, 2), (4, -1), (5, 0), (2, ODD)])


def test_binding_refusals(q):
    """The binding refuses host tensors, and shapes and types before any call."""
    cpu = torch.zeros((2, 4))
    for call in (lambda: q.moe_route(cpu, 2), lambda: q.swiglu(cpu), lambda: q.moe_sort(cpu.int(), 4),
                 lambda: q.moe_gather(cpu, cpu.int()), lambda: q.moe_combine(cpu, cpu.int()),
                 lambda: q.int4_gemm(cpu.to(torch.uint8), cpu.bfloat16(), cpu.bfloat16())):
        with pytest.raises(ValueError):
            call()
