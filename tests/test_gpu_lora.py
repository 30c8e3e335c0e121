"""GPU parity of the low-rank adapters and their gradients against the float64 oracle.

Tolerances, with u = 2^-24: z is a float32 sum of K products, off by (K + 8) u times the sum of magnitudes;
it goes on in pieces that hold 24 bits (float32 results) or 16 (bfloat16: 2^-16 of it), and the second sum has at most
3 R terms: (K + 3 R + 32) u B, and 2^-16 B for bfloat16, B the sum of magnitudes behind the result.  A bfloat16
result adds half a step, 2^-8; `base` adds u of itself."""

import numpy as np
import pytest
import torch

from oracle import block as O
from gpu_util import DEV, show

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
PIECES = {torch.float32: U, torch.bfloat16: 2.0 ** -16}


@pytest.fixture(scope="module")
def q():
    import weight_quantized_linear_amd as q
    return q


def f64(t):
    return t.double().cpu().numpy()


def random(rng, shape, dtype=torch.bfloat16, std=1.0):
    return torch.from_numpy(rng.normal(size=shape) * std).to(dtype).to(DEV)


def offset(t, by=1):
    flat = torch.full((t.numel() + by + 8,), float("nan"), dtype=t.dtype, device=DEV)
    flat[by:by + t.numel()] = t.reshape(-1)
    return flat[by:by + t.numel()].view(t.shape)


def close(out, ref, tau, dtype):
    err = np.abs(f64(out) - ref)
    ok = err <= tau + HALF[dtype] * (np.abs(ref) + tau) + 2.0 ** -126
    if not ok.all():
        at = np.unravel_index(np.argmax(np.where(ok, 0, err / (tau + 1e-300))), ok.shape)
        print("worst at", at, "out", f64(out)[at], "ref", ref[at], "tau", tau[at], "bad", (~ok).sum(), "of", ok.size)
    return bool(ok.all())


def groups(rng, counts, adapters, lead=0):
    """Offsets from `lead` on, and an adapter for each group, every fifth with none."""
    off = np.concatenate([[lead], lead + np.cumsum(counts)]).astype(np.int32)
    ids = rng.integers(0, adapters, len(counts)).astype(np.int32)
    ids[4::5] = rng.choice([-1, adapters, -7])
    return off, ids


def check(q, rng, counts, adapters, r, k, n, out_dtype, base, lead=0, tail=0, odd=False, scaled=True):
    t = lead + int(np.sum(counts)) + tail
    show("lora", t, len(counts), adapters, r, k, n, out_dtype, base, odd)
    off, ids = groups(rng, counts, adapters, lead)
    x, a, b = random(rng, (t, k)), random(rng, (adapters, r, k), std=k ** -0.5), random(rng, (adapters, n, r), std=r ** -0.5)
    s = torch.from_numpy(rng.uniform(0.5, 2.0, adapters)).float().to(DEV) if scaled else None
    bt = random(rng, (t, n), out_dtype) if base else None
    dy, dx0 = random(rng, (t, n)), random(rng, (t, k), out_dtype) if base else None
    if odd:
        x, a, b, dy = offset(x), offset(a), offset(b), offset(dy)
        bt, dx0 = (offset(bt), offset(dx0)) if base else (None, None)
    offs, idt = torch.from_numpy(off).to(DEV), torch.from_numpy(ids).to(DEV)
    s64 = f64(s) if scaled else np.ones(adapters)
    x64, a64, b64 = f64(x), f64(a), f64(b)

    room = torch.full((t * n + 16,), 7.0, dtype=out_dtype, device=DEV)
    out = room[8 - odd:8 - odd + t * n].view(t, n)
    got, z = q.lora_gemm(x, a, b, offs, idt, scale=s, base=bt, out=out, out_dtype=out_dtype, return_z=True)
    again = q.lora_gemm(x, a, b, offs, idt, scale=s, base=bt, out=torch.full_like(out, 7.0), out_dtype=out_dtype)
    ref, zref, bound, zbound, written = O.lora(x64, a64, b64, off, ids, s64, f64(bt) if base else None, n)
    assert bool((room[:8 - odd] == 7).all()) and bool((room[8 - odd + t * n:] == 7).all()), "writes outside out"
    assert torch.equal(got, again), "two runs differ"
    assert bool((got[torch.from_numpy(~written).to(DEV)] == 7).all()), "rows in no group"
    assert close(z[torch.from_numpy(written).to(DEV)], zref[written], (k + 8) * U * zbound[written], torch.float32), "z"
    tau = ((k + 3 * r + 32) * U + PIECES[out_dtype]) * bound + (U * np.abs(f64(bt)) if base else 0.0)
    assert close(got[torch.from_numpy(written).to(DEV)], ref[written], tau[written], out_dtype), "out"

    z64 = f64(z)
    for param in (torch.float32, torch.bfloat16):
        buf = torch.full((t, k), 7.0, dtype=out_dtype, device=DEV)
        dx, da, db = q.lora_gemm_backward(dy, x, z, a, b, offs, idt, scale=s, base=dx0, grad_x=buf, grad_x_dtype=out_dtype,
                                          param_dtype=param)
        z64[~written] = 0.0
        rx, ra, rb, xb, ab, bb = O.lora_backward(f64(dy), x64, z64, a64, b64, off, ids, s64, f64(dx0) if base else None)
        assert bool((dx[torch.from_numpy(~written).to(DEV)] == 7).all()), "rows in no group"
        tau = ((n + 3 * r + 32) * U + PIECES[out_dtype]) * xb + (U * np.abs(f64(dx0)) if base else 0.0)
        assert close(dx[torch.from_numpy(written).to(DEV)], rx[written], tau[written], out_dtype), "dx"
        assert close(da, ra, ((n + 3 * t + 32) * U + PIECES[param]) * ab, param), "da"
        assert close(db, rb, ((3 * t + 32) * U + PIECES[param]) * bb, param), "db"


CASES = [  # counts, adapters, r, k, n
    ([1], 1, 1, 1, 1),
    ([1] * 9, 4, 16, 128, 128),
    ([3, 0, 5, 1, 2], 2, 8, 64, 72),
    ([1, 2, 40, 7, 1, 0, 17], 3, 4, 100, 33),
    ([16, 17, 15, 33], 4, 16, 256, 64),
    ([64, 1, 65, 130], 5, 64, 320, 264),
    ([200], 1, 32, 512, 136),
    ([5, 90, 3], 2, 100, 200, 80),
    ([70, 30], 3, 128, 136, 72),
    ([9, 80], 1, 256, 264, 40),
    ([33, 34, 35], 2, 7, 63, 65),
    ([40, 3], 2, 12, 5, 6),
    ([20], 1, 16, 7, 300),
    ([70, 2], 2, 9, 301, 3),
    ([130, 66], 2, 33, 1030, 2001),
]


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("base", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_lora(q, out_dtype, base, case):
    counts, adapters, r, k, n = CASES[case]
    rng = np.random.default_rng([1, case, base])
    check(q, rng, counts, adapters, r, k, n, out_dtype, base, lead=case % 3, tail=case % 4, scaled=case % 2 == 0)


@pytest.mark.parametrize("case", [1, 2, 4, 5, 8])
def test_lora_off_alignment(q, case):
    counts, adapters, r, k, n = CASES[case]
    check(q, np.random.default_rng([2, case]), counts, adapters, r, k, n, torch.bfloat16, True, odd=True)


@pytest.mark.parametrize("counts,adapters,r,k,n", [([1] * 64, 32, 16, 4096, 2048), ([300, 1, 800, 25, 900], 3, 64, 2048, 1024),
                                                   ([1500], 1, 16, 1024, 2048), ([700, 900], 2, 200, 512, 520)])
def test_lora_large(q, counts, adapters, r, k, n):
    check(q, np.random.default_rng([3, r, k]), counts, adapters, r, k, n, torch.bfloat16, True)


def test_more_groups_than_a_wave(q):
    rng = np.random.default_rng(4)
    check(q, rng, rng.integers(0, 4, 300), 7, 8, 64, 40, torch.float32, True)
    check(q, rng, rng.integers(0, 2, 4096), 40, 4, 32, 16, torch.float32, True)


def test_in_place(q):
    rng = np.random.default_rng(5)
    off, ids = groups(rng, [5, 20, 9], 2)
    offs, idt = torch.from_numpy(off).to(DEV), torch.from_numpy(ids).to(DEV)
    x, a, b = random(rng, (34, 64)), random(rng, (2, 8, 64)), random(rng, (2, 48, 8))
    base, dy, dx0 = random(rng, (34, 48)), random(rng, (34, 48)), random(rng, (34, 64))
    want, z = q.lora_gemm(x, a, b, offs, idt, base=base, return_z=True)
    got = base.clone()
    assert torch.equal(q.lora_gemm(x, a, b, offs, idt, base=got, out=got), want)
    wx, wa, wb = q.lora_gemm_backward(dy, x, z, a, b, offs, idt, base=dx0)
    buf = dx0.clone()
    gx, ga, gb = q.lora_gemm_backward(dy, x, z, a, b, offs, idt, base=buf, grad_x=buf)
    assert torch.equal(gx, wx) and torch.equal(ga, wa) and torch.equal(gb, wb)


def test_offsets_past_the_rows_and_falling(q):
    """Offsets are clipped to T; where they fall, results are undefined but nothing outside is touched."""
    rng = np.random.default_rng(6)
    x, a, b = random(rng, (20, 32)), random(rng, (2, 8, 32)), random(rng, (2, 24, 8))
    ids = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    want = q.lora_gemm(x, a, b, torch.tensor([0, 7, 20], dtype=torch.int32, device=DEV), ids)
    got = q.lora_gemm(x, a, b, torch.tensor([0, 7, 2 ** 30], dtype=torch.int32, device=DEV), ids)
    assert torch.equal(got, want)
    for off in ([0, 15, 4], [18, 3, 20], [-1, -1, -1], [25, 3, 30]):
        o = torch.tensor(off, dtype=torch.int32, device=DEV)
        room = torch.full((22, 24), 7.0, dtype=torch.bfloat16, device=DEV)
        _, z = q.lora_gemm(x, a, b, o, ids, out=room[1:21], return_z=True)
        q.lora_gemm_backward(room[1:21].nan_to_num(), x, z.nan_to_num(), a, b, o, ids)
        torch.cuda.synchronize()
        assert bool((room[0] == 7).all()) and bool((room[21] == 7).all())


def test_not_finite_stays_in_its_rows(q):
    rng = np.random.default_rng(7)
    off, ids = torch.tensor([0, 3, 6], dtype=torch.int32, device=DEV), torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    x, a, b = random(rng, (6, 32)), random(rng, (2, 8, 32)), random(rng, (2, 24, 8))
    x[4, 3], x[1, 0] = float("nan"), float("inf")
    out, z = q.lora_gemm(x, a, b, off, ids, return_z=True)
    bad = ~out.isfinite().all(1)
    assert bad.tolist() == [False, True, False, False, True, False]
    _, da, db = q.lora_gemm_backward(random(rng, (6, 24)), x[:].nan_to_num(0.0, 0.0, 0.0), z.nan_to_num(0.0, 0.0, 0.0), a, b, off, ids)
    assert bool(da.isfinite().all()) and bool(db.isfinite().all())
    # the largest finite values keep finite pieces
    big = torch.full((1, 8), 3.3e38, dtype=torch.bfloat16, device=DEV)
    one = torch.zeros((1, 1, 8), dtype=torch.bfloat16, device=DEV)
    one[0, 0, 0] = 1.0
    o = q.lora_gemm(big, one, torch.full((1, 8, 1), 0.5, dtype=torch.bfloat16, device=DEV),
                    torch.tensor([0, 1], dtype=torch.int32, device=DEV), torch.tensor([0], dtype=torch.int32, device=DEV),
                    out_dtype=torch.float32)
    assert bool((o == 0.5 * big.float()[0, 0]).all())


def test_empty(q):
    x, a, b = (torch.ones(s, dtype=torch.bfloat16, device=DEV) for s in ((0, 32), (2, 8, 32), (2, 24, 8)))
    off, ids = torch.zeros(2, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    out, z = q.lora_gemm(x, a, b, off, ids, return_z=True)
    assert out.shape == (0, 24) and z.shape == (0, 8)
    dx, da, db = q.lora_gemm_backward(out, x, z, a, b, off, ids)
    assert dx.shape == (0, 32) and not da.any() and not db.any()
