"""Grouped FP8, NVFP4 and int8 products over offsets that fall and rise again: thousands of
groups would cover the same rows.  The first one does; the result of the others is undefined, the
reads and writes are not.  Inputs are small integers, so every sum is exact."""

import pytest
import torch

from gpu_util import DEV, show

pytestmark = pytest.mark.gpu

N, K, E = 16, 64, 3


@pytest.fixture(scope="module")
def q():
    import weight_quantized_linear_amd as q
    return q


def falling(groups):
    """0, the largest offset, 0, ...: every other group covers all rows."""
    offs = torch.tensor([0, -1], dtype=torch.int32, device=DEV).repeat(groups // 2 + 1)[:groups + 1].contiguous()
    return offs, torch.full((groups,), 1, dtype=torch.int32, device=DEV)


def guarded(t, dtype, fill):
    buf = torch.full((t + 2000, N), fill, dtype=dtype, device=DEV)
    return buf, buf[1000:1000 + t]


def check(buf, out, fill, want):
    assert torch.all(buf[:1000] == fill) and torch.all(buf[1000 + out.shape[0]:] == fill)
    assert bool((out.view(-1, 1000, N) == want.to(out.dtype)).all())


def integers(t, dtype):
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randint(-4, 5, (1000, K), generator=g, device=DEV)
    return x.double(), x.to(dtype).repeat(t // 1000, 1)


def test_fp8(q):
    t, groups = 33_000_000, 8600
    ref, x = integers(t, torch.bfloat16)
    w = torch.randint(-4, 5, (E, N, K), device=DEV).float().to(torch.float8_e4m3fn)
    buf, out = guarded(t, torch.bfloat16, 7.0)
    show("fp8 falling offsets", t, groups)
    q.fp8_grouped_gemm(w, x, *falling(groups), out=out)
    check(buf, out, 7.0, ref @ w[1].double().t().contiguous())


def test_nvfp4(q):
    t, groups = 33_000_000, 8600
    ref, x = integers(t, torch.bfloat16)
    w = torch.randint(0, 256, (E, N, K // 2), device=DEV, dtype=torch.uint8)
    s = torch.ones((E, N, K // 16), device=DEV).to(torch.float8_e4m3fn)
    buf, out = guarded(t, torch.bfloat16, 7.0)
    show("nvfp4 falling offsets", t, groups)
    q.nvfp4_grouped_gemm(w, s, x, *falling(groups), out=out)
    check(buf, out, 7.0, ref @ q.nvfp4_dequant(w[1].contiguous(), s[1].contiguous()).double().t().contiguous())


def test_int8(q):
    t, groups = 34_000_000, 8192
    ref, a = integers(t, torch.int8)
    b = torch.randint(-100, 101, (E, N, K), device=DEV).to(torch.int8)
    buf, out = guarded(t, torch.int32, 7)
    show("int8 falling offsets", t, groups)
    q.int8_grouped_gemm(a, b, None, None, *falling(groups), out=out, out_dtype=torch.int32)
    check(buf, out, 7, ref @ b[1].double().t().contiguous())
