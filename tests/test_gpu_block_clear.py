"""Parameter gradients of a call without rows are cleared at any size, here with more 2-byte values than a launch
has threads (2^32)."""

import pytest
import torch

from gpu_util import DEV, show

pytestmark = pytest.mark.gpu


def test_gradients_without_rows_past_8_gib():
    import weight_quantized_linear_amd as q
    n, k = 46400, 46340
    assert n * k * 4 // 2 > 1 << 32
    show("grad_w without rows", n, k)
    grad = torch.full((n, k), 7.0, device=DEV)
    p, s = grad.data_ptr(), torch.cuda.current_stream().cuda_stream
    assert q.lib.qlinear_bf16_gemm_grad_w(p, p, p, q.F32, 0, n, k, None, 0, s) == q.OK
    assert int(torch.count_nonzero(grad)) == 0
