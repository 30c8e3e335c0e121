"""A grid has fewer than 2^32 threads along an axis: a call that would need more is refused and writes nothing, and
the largest grid below that is whole."""

import pytest
import torch

from gpu_util import DEV, show

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import weight_quantized_linear_amd as q
    return q


@pytest.mark.parametrize("rows,fits", [((1 << 30) - 64, True), ((1 << 30) + 1, False)])
def test_rows_at_the_limit(q, rows, fits):
    """Tiles of 64 rows and 256 threads: 2^30 rows are 2^32 threads."""
    show("launch limit", rows)
    dout = torch.full((rows, 1), 2.0, dtype=torch.bfloat16, device=DEV)
    w = torch.full((1, 1), 3.0, dtype=torch.bfloat16, device=DEV)
    out = torch.full((rows, 1), 7.0, dtype=torch.bfloat16, device=DEV)
    if fits:
        q.bf16_gemm_grad_x(dout, w, out=out)
        assert bool((out == 6).all())
    else:
        with pytest.raises(q.QLinearError) as e:
            q.bf16_gemm_grad_x(dout, w, out=out)
        assert e.value.status == q.ERR_LAUNCH
        assert bool((out == 7).all())
