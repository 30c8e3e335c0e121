"""A mixture-of-experts feed-forward layer with int4 experts, from the library's calls.

    router logits -> moe_route -> moe_sort -> moe_gather
        -> int4_grouped_gemm (gate and up) -> swiglu -> int4_grouped_gemm (down) -> moe_combine

and the gradients that training a router in front of frozen int4 experts takes: the
loss reaches the logits through the weights of the sum (moe_combine_backward,
moe_route_backward).  Run it to see both against a plain float32 layer:

    python examples/moe_layer.py
"""

from __future__ import annotations

import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_quantized_linear_amd as q  # noqa: E402


def quantize_int4(w: torch.Tensor, group: int):
    """Codes, scales and zero points of [..., N, K] weights, one pair per `group` values of k.
    A group's range takes in 0, which the zero point 0 .. 15 has to stand for."""
    k = w.shape[-1]
    g = w.float().unflatten(-1, (k // group, group))
    low, high = g.amin(-1).clamp(max=0.0), g.amax(-1).clamp(min=0.0)
    scale = ((high - low) / 15.0).clamp(min=1e-8).bfloat16()
    zero = (-low / scale.float()).round().clamp(0, 15)
    codes = (g / scale.float()[..., None] + zero[..., None]).round().clamp(0, 15).flatten(-2).to(torch.uint8)
    return (codes[..., 0::2] | codes[..., 1::2] << 4).contiguous(), scale.contiguous(), zero.to(torch.uint8).contiguous()


def dequantize_int4(packed, scale, zero, group: int):
    codes = torch.stack([packed & 15, packed >> 4], -1).flatten(-2).float()
    return (codes - zero.float().repeat_interleave(group, -1)) * scale.float().repeat_interleave(group, -1)


@dataclass
class Saved:
    """What a forward pass keeps for the router's gradient."""
    logits: torch.Tensor
    ids: torch.Tensor
    weights: torch.Tensor
    slot_row: torch.Tensor
    rows: torch.Tensor


class MoeLayer:
    def __init__(self, router: torch.Tensor, gate_up: torch.Tensor, down: torch.Tensor, top_k: int, group: int = 128):
        """router [E, H] float32, gate_up [E, 2F, H], down [E, H, F]."""
        self.router, self.top_k, self.group = router, top_k, group
        self.gate_up, self.down = quantize_int4(gate_up, group), quantize_int4(down, group)
        self.num_experts = router.shape[0]
        self.every = torch.arange(self.num_experts, dtype=torch.int32, device=router.device)

    def _experts(self, weight, rows, offsets):
        w, scale, zero = weight
        return q.int4_grouped_gemm(w, scale, rows, offsets, self.every, w_zero=zero, group_size=self.group)

    def forward(self, x: torch.Tensor):
        """x [T, H] bfloat16 -> (y [T, H], what the gradient needs)."""
        logits = x.float() @ self.router.t()
        ids, weights = q.moe_route(logits, self.top_k)
        offsets, _, slot_row = q.moe_sort(ids, self.num_experts)
        hidden = q.swiglu(self._experts(self.gate_up, q.moe_gather(x, slot_row), offsets))
        rows = self._experts(self.down, hidden, offsets)
        return q.moe_combine(rows, slot_row, weights), Saved(logits, ids, weights, slot_row, rows)

    def router_gradient(self, grad_y: torch.Tensor, x: torch.Tensor, s: Saved) -> torch.Tensor:
        """Gradient of the router [E, H] through the experts' weights."""
        _, grad_weights = q.moe_combine_backward(grad_y, s.rows, s.slot_row, s.weights)
        return q.moe_route_backward(s.logits, s.ids, grad_weights).t() @ x.float()


def plain(layer: MoeLayer, x: torch.Tensor, grad_y: torch.Tensor):
    """The same layer in float32, every expert over every token; (y, the router's gradient)."""
    gate_up = dequantize_int4(*layer.gate_up, layer.group)
    down = dequantize_int4(*layer.down, layer.group)
    router = layer.router.clone().requires_grad_(True)
    xf = x.float()
    logits = xf @ router.t()
    p, ids = logits.softmax(1).topk(layer.top_k, 1)
    weights = p / p.sum(1, keepdim=True)
    y = torch.zeros_like(xf)
    for e in range(layer.num_experts):
        gate, up = (xf @ gate_up[e].t()).chunk(2, 1)
        part = (torch.nn.functional.silu(gate) * up) @ down[e].t()
        y = y + part * torch.where(ids == e, weights, 0.0).sum(1, keepdim=True)
    y.backward(grad_y.float())
    return y.detach(), router.grad


def run(tokens: int, hidden: int = 512, inner: int = 384, experts: int = 16, top_k: int = 4, seed: int = 0):
    """(relative distance of y, of the router's gradient) to the plain layer's."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda") * std

    layer = MoeLayer(normal(experts, hidden, std=hidden ** -0.5), normal(experts, 2 * inner, hidden, std=hidden ** -0.5),
                     normal(experts, hidden, inner, std=inner ** -0.5), top_k)
    x, grad_y = normal(tokens, hidden).bfloat16(), normal(tokens, hidden).bfloat16()
    y, saved = layer.forward(x)
    grad = layer.router_gradient(grad_y, x, saved)
    want_y, want_grad = plain(layer, x, grad_y)

    def distance(a, b):
        return float((a.float() - b).norm() / b.norm())

    return distance(y, want_y), distance(grad, want_grad)


if __name__ == "__main__":
    for n in (1, 8, 200, 3000):
        y, grad = run(n)
        print(f"{n:5d} tokens: output {y:.2e}, router gradient {grad:.2e} from the float32 layer", flush=True)
