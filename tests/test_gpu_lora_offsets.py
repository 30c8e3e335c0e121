"""Adapters' gradients over offsets that fall: the results are those of the groups that have rows in the forward
pass, a group that begins before an earlier one's end has none, and no other row is looked at."""

import ctypes

import pytest
import torch

from gpu_util import DEV, show

pytestmark = pytest.mark.gpu

T, K, N, R, L = 20, 32, 24, 8, 2


@pytest.fixture(scope="module")
def q():
    import weight_quantized_linear_amd as q
    return q


def offsets(groups, fall):
    """`groups` groups: rows 0 .. 14, empty ones, then a fall to 4 and a group 4 .. 19 as group `fall`."""
    off = [0] + [15] * groups
    off[fall] = 4
    off[fall + 1] = T
    for z in range(fall + 2, groups + 1):
        off[z] = T
    return off


@pytest.mark.parametrize("groups,fall", [(3, 2), (64, 63), (70, 64), (70, 66), (200, 130)])
@pytest.mark.parametrize("param_dtype", [torch.float32, torch.bfloat16])
def test_dropped_groups_have_no_gradient(q, groups, fall, param_dtype):
    show("lora gradients, falling offsets", groups, fall, param_dtype)
    g = torch.Generator(device=DEV).manual_seed(groups + fall)
    x, a, b, dy = (torch.randn(s, generator=g, device=DEV).to(torch.bfloat16)
                   for s in ((T, K), (L, R, K), (L, N, R), (T, N)))
    ids = torch.ones(groups, dtype=torch.int32, device=DEV)
    ids[0] = 0
    off = torch.tensor(offsets(groups, fall), dtype=torch.int32, device=DEV)
    kept = torch.tensor([0] + [15] * groups, dtype=torch.int32, device=DEV)
    _, z = q.lora_gemm(x, a, b, kept, ids, return_z=True)
    z[15:] = float("nan")  # as the forward pass leaves them: not written
    need = ctypes.c_int64(0)
    assert q.lib.qlinear_lora_backward_workspace_size(groups, L, T, N, K, R, ctypes.byref(need)) == 0
    results = []
    for o in (off, kept):
        ws = torch.full(((need.value + 3) // 4 + 4,), float("nan"), device=DEV)
        dx = torch.full((T, K), 7.0, dtype=torch.bfloat16, device=DEV)
        results.append(q.lora_gemm_backward(dy, x, z, a, b, o, ids, grad_x=dx, param_dtype=param_dtype, workspace=ws))
    (dx, da, db), (wx, wa, wb) = results
    assert bool(da.isfinite().all()) and bool(db.isfinite().all())
    assert torch.equal(da, wa) and torch.equal(db, wb) and torch.equal(dx, wx)
    assert not da[1].any() and not db[1].any() and bool((dx[15:] == 7).all())
