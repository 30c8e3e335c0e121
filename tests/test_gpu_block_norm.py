"""GPU parity of the block norm and its gradients against the float64 oracle.

Tolerances, with u = 2^-24: the mean of H squares is off by (H + 4) u of itself, its inverse root by half that
and 4 u, so a normed value by (H / 2 + 16) u; residual_out by that of the gated part and 4 u of both parts.
`out` is held to the formula on residual_out as it was stored.  The gradients add sums of H terms over the row
and of T terms over the rows: (2 H + 32) u and (T + 2 H + 32) u of the sums of magnitudes behind them.  A result
in bfloat16 adds half a step, 2^-8."""

import numpy as np
import pytest
import torch

from oracle import block as O
from gpu_util import DEV, show

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
F, B = torch.float32, torch.bfloat16
TYPES = [(B, B, B), (B, B, F), (F, B, B), (F, B, F), (F, F, B), (F, F, F)]  # residual, block, parameters


@pytest.fixture(scope="module")
def q():
    import weight_quantized_linear_amd as q
    return q


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def offset(t, by=1):
    flat = torch.full((t.numel() + by + 8,), float("nan"), dtype=t.dtype, device=DEV)
    flat[by:by + t.numel()] = t.reshape(-1)
    return flat[by:by + t.numel()].view(t.shape)


def close(name, out, ref, tau, dtype):
    err = np.abs(f64(out) - ref)
    ok = err <= tau + HALF[dtype] * (np.abs(ref) + tau) + 2.0 ** -126
    if not ok.all():
        at = np.unravel_index(np.argmax(np.where(ok, 0, err / (tau + 1e-300))), ok.shape)
        print(name, "worst at", at, "out", f64(out)[at], "ref", ref[at], "tau", tau[at], "bad", (~ok).sum(), "of", ok.size)
    return bool(ok.all())


def check(q, t, h, types, post, gates, scale=1.0, eps=1e-6, with_block=True, odd=False, grad_in=True, std=1.0):
    rt, bt, pt = types
    show("norm", t, h, types, post, gates, scale, with_block, odd)
    rng = np.random.default_rng([t, h, post, gates])
    put = offset if odd else lambda v: v

    def random(shape, dtype, std=1.0, mean=0.0):
        return put(torch.from_numpy(rng.normal(size=shape) * std + mean).to(dtype).to(DEV))

    res, w = random((t, h), rt, std), random((h,), pt, 0.3, 1.0)
    block = random((t, h), bt, 2.0) if with_block else None
    wo = random((h,), pt, 0.3, 1.0) if post else None
    gate = random((gates, h), pt) if gates else None
    kw = dict(block=block, block_weight=wo, gate=gate, residual_scale=scale, eps=eps)
    room = torch.full((t * h + 16,), 7.0, dtype=bt, device=DEV)
    start = 1 if odd else 8
    out = room[start:start + t * h].view(t, h)
    y, r2 = q.block_norm(res, w, out=out, **({} if with_block else {"out_dtype": bt}), **kw)
    assert bool((room[:start] == 7).all()) and bool((room[start + t * h:] == 7).all()), "writes outside out"
    eps64, scale64 = float(np.float32(eps)), float(np.float32(scale))
    ref, rr = O.norm(f64(res), f64(w), f64(block), f64(wo), f64(gate), scale64, eps64, lambda v: f64(r2))
    if with_block:
        p = O.norm(np.zeros((t, h)), f64(w), f64(block), f64(wo), f64(gate), 1.0, eps64, lambda v: v)[1]
        assert close("res", r2, rr, 4 * U * np.abs(scale64 * f64(res)) + (h / 2 + 20) * U * np.abs(p), rt)
    else:
        assert r2 is res
    assert close("out", y, ref, (h / 2 + 16) * U * np.abs(ref), bt)

    dy, dr = random((t, h), bt), random((t, h), rt) if grad_in else None
    g = q.block_norm_backward(dy, dr, r2, w, **kw)
    n = O.norm_backward(f64(dy), f64(dr), f64(r2), f64(w), f64(block), f64(wo), f64(gate), scale64, eps64)
    row, col = (2 * h + 32) * U, (t + 2 * h + 32) * U
    assert close("dres", g.residual, n["residual"], row * n["residual_bound"], rt)
    assert close("dw", g.weight, n["weight"], col * n["weight_bound"], pt)
    if with_block:
        assert close("dblock", g.block, n["block"], 2 * row * n["block_bound"], bt)
    else:
        assert g.block is None
    assert (g.block_weight is None) == (not post) and (g.gate is None) == (not gates)
    if post:
        assert close("dwo", g.block_weight, n["block_weight"], 2 * col * n["block_weight_bound"], pt)
    if gates:
        assert close("dgate", g.gate, n["gate"], 2 * col * n["gate_bound"], pt)
    again = q.block_norm_backward(dy, dr, r2, w, **kw)
    for a, b in zip(g, again):
        assert (a is None and b is None) or torch.equal(a, b), "two runs differ"


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("t,h,gates", [(1, 1, 0), (2, 7, 1), (6, 64, 3), (5, 100, 5), (9, 512, 0), (12, 1000, 4), (7, 2048, 1),
                                       (3, 4096, 3), (4, 3001, 2)])
def test_block_norm(q, types, post, t, h, gates):
    check(q, t, h, types, post, gates, scale=0.5 if gates == 1 else 1.0)


@pytest.mark.parametrize("gates", [0, 1, 2, 4, 5, 13, 20, 52, 80, 260, 520, 1040])
def test_gates_over_many_rows(q, gates):
    """Gates whose rows end inside, at and across the ranges of rows that one worker sums."""
    check(q, 1040, 1040, (B, B, F), True, gates)
    check(q, 1040, 2056, (F, F, F), False, gates)


@pytest.mark.parametrize("h", [511, 513, 1023, 1024, 1025, 2049, 4097, 8192, 8200, 16383, 16384])
@pytest.mark.parametrize("types", [(B, B, B), (F, F, F)])
def test_widths(q, h, types):
    check(q, 5, h, types, True, 1)


@pytest.mark.parametrize("t", [1, 2, 3, 255, 511, 512, 513, 2047, 2049, 5000])
def test_row_counts(q, t):
    check(q, t, 72, (B, B, F), True, 1)
    check(q, t, 72, (F, B, F), True, t)


@pytest.mark.parametrize("types", [(B, B, B), (F, F, F), (F, B, F)])
def test_off_alignment(q, types):
    check(q, 6, 256, types, True, 3, odd=True)
    check(q, 6, 1100, types, False, 0, odd=True)


@pytest.mark.parametrize("types", [(B, B, F), (F, B, B), (F, F, F)])
@pytest.mark.parametrize("t,h", [(1, 16), (33, 520), (700, 96), (9, 5000)])
def test_plain_norm(q, types, t, h):
    check(q, t, h, types, False, 0, with_block=False, scale=0.25)
    check(q, t, h, types, False, 0, with_block=False, grad_in=False)


@pytest.mark.parametrize("std", [1e-12, 1e-3, 1e12])
def test_magnitudes(q, std):
    check(q, 4, 300, (F, F, F), True, 1, std=std, eps=1e-5)


def test_zero_rows_and_no_outer_gradient(q):
    check(q, 5, 300, (B, B, F), True, 1, grad_in=False)
    z = torch.zeros((2, 64), device=DEV)
    w = torch.ones(64, device=DEV)
    y, r = q.block_norm(z, w, block=z, block_weight=w)
    assert not y.any() and not r.any()
    g = q.block_norm_backward(z + 1.0, None, z, w, block=z, block_weight=w, eps=1.0)
    assert torch.equal(g.residual, z + 1.0) and not g.weight.any() and torch.equal(g.block, z + 1.0)


def test_in_place(q):
    rng = np.random.default_rng(3)
    res, block, dy, dr = (torch.from_numpy(rng.normal(size=(40, 520))).to(B).to(DEV) for _ in range(4))
    w = torch.ones(520, dtype=B, device=DEV)
    y, r = q.block_norm(res, w, block=block, block_weight=w)
    buf = res.clone()
    y2, r2 = q.block_norm(buf, w, block=block, block_weight=w, residual_out=buf)
    assert r2.data_ptr() == buf.data_ptr() and torch.equal(y, y2) and torch.equal(r, r2)
    g = q.block_norm_backward(dy, dr, r, w, block=block, block_weight=w)
    buf = dr.clone()
    g2 = q.block_norm_backward(dy, buf, r, w, block=block, block_weight=w, grad_residual=buf)
    assert torch.equal(g.residual, g2.residual) and torch.equal(g.block, g2.block)


def test_empty(q):
    res, w, gate = torch.zeros((0, 64), device=DEV), torch.ones(64, device=DEV), torch.ones((3, 64), device=DEV)
    y, r = q.block_norm(res, w, block=res, block_weight=w, gate=gate)
    assert y.shape == (0, 64) and r.shape == (0, 64)
    g = q.block_norm_backward(y, None, r, w, block=res, block_weight=w, gate=gate)
    assert not g.weight.any() and not g.block_weight.any() and not g.gate.any() and g.gate.shape == (3, 64)


def test_not_finite_stays_in_its_row(q):
    res = torch.ones((4, 96), device=DEV)
    res[2, 5] = float("nan")
    w = torch.ones(96, device=DEV)
    y, _ = q.block_norm(res, w)
    assert y.isnan().any(1).tolist() == [False, False, True, False] and bool(y[2].isnan().all())
