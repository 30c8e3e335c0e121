"""Operands that are not contiguous are refused by every call of the feed-forward block, before any device work."""

import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu

T, K, N, R, L, H = 6, 32, 24, 8, 2, 32


def strided(t):
    """The same values in a tensor of the same shape whose memory has gaps."""
    wide = torch.zeros((*t.shape[:-1], 2 * t.shape[-1]), dtype=t.dtype, device=DEV)
    view = wide[..., ::2]
    view.copy_(t)
    return view


def bf(*shape):
    return torch.ones(shape, dtype=torch.bfloat16, device=DEV)


def calls(q):
    off, ids = torch.tensor([0, 2, T], dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)
    adapters = dict(x=bf(T, K), a=bf(L, R, K), b=bf(L, N, R), a_offsets=off, adapter_ids=ids, scale=torch.ones(L, device=DEV))
    return {
        q.gated_gemm: dict(w=bf(2 * N, K), x=bf(T, K), addend=bf(T, 2 * N), out=bf(T, N)),
        q.gated_gemm_backward: dict(grad_out=bf(T, N), pre=bf(T, 2 * N), w=bf(2 * N, K), x=bf(T, K)),
        q.bf16_gemm_grad_x: dict(grad_out=bf(T, N), w=bf(N, K), out=bf(T, K), workspace=ws),
        q.bf16_gemm_grad_w: dict(grad_out=bf(T, N), x=bf(T, K), out=bf(N, K), workspace=ws),
        q.lora_gemm: dict(adapters, base=bf(T, N), out=bf(T, N), workspace=ws),
        q.lora_gemm_backward: dict(adapters, grad_out=bf(T, N), z=torch.ones((T, R), device=DEV), base=bf(T, K), grad_x=bf(T, K),
                                   workspace=ws),
        q.block_norm: dict(residual=bf(T, H), weight=bf(H), block=bf(T, H), block_weight=bf(H), gate=bf(2, H), out=bf(T, H),
                           residual_out=bf(T, H)),
        q.block_norm_backward: dict(grad_out=bf(T, H), grad_residual_out=bf(T, H), residual_out=bf(T, H), weight=bf(H), block=bf(T, H),
                                    block_weight=bf(H), gate=bf(2, H), grad_residual=bf(T, H), workspace=ws),
    }


def test_strided_operands():
    import weight_quantized_linear_amd as q
    for call, operands in calls(q).items():
        call(**operands)
        for name, t in operands.items():
            kept = t.clone()
            with pytest.raises(ValueError, match="contiguous"):
                call(**{**operands, name: strided(t)})
            assert torch.equal(t, kept), (call.__name__, name)
