"""The gated product's backward pass has no alpha in its products: a call that says it had one is refused where
they are needed, and makes grad_pre otherwise (CPU only)."""

import pytest
import torch

from test_block_arguments import bf, q, recorder  # noqa: F401 (fixtures)


@pytest.mark.parametrize("need", [dict(), dict(need_w=False), dict(need_x=False)])
@pytest.mark.parametrize("factors", [dict(alpha=0.5), dict(alpha_up=2.0), dict(alpha=0.5, alpha_up=1.0), dict(alpha=float("nan"))])
def test_alpha_is_refused_where_a_product_is_needed(q, recorder, need, factors):  # noqa: F811
    with pytest.raises(ValueError, match="alpha"):
        q.gated_gemm_backward(bf(3, 8), bf(3, 16), bf(16, 32), bf(3, 32), **need, **factors)
    assert recorder.name is None


def test_grad_pre_alone_takes_any_alpha(q, recorder):  # noqa: F811
    g, dx, dw = q.gated_gemm_backward(bf(3, 8), bf(3, 16), bf(16, 32), bf(3, 32), need_x=False, need_w=False, alpha=0.5, alpha_up=2.0)
    assert recorder.name == "qlinear_gated_backward" and dx is None and dw is None and g.shape == (3, 16)
