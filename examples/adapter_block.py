"""A feed-forward block of a transformer with low-rank adapters, from the library's calls.

    block_norm (end of the block before, norm in front of this one)
        -> gated_gemm (gate and up projection with their adapters' part as the addend)
        -> bf16_gemm (down projection) -> lora_gemm (its adapters, added in place)

The rows are those of several requests, each with an adapter of its own or with none, and the
projections are shared.  ``backward`` gives what training the adapters and the norms on frozen
projections takes.  Run it to see the output and all gradients against a plain float32 block:

    python examples/adapter_block.py
"""

from __future__ import annotations

import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_quantized_linear_amd as q  # noqa: E402


@dataclass
class Requests:
    """Rows offsets[y] .. offsets[y + 1] - 1 belong to request y, with adapter ids[y] (-1: none).
    The requests cover all rows."""
    offsets: torch.Tensor
    ids: torch.Tensor


@dataclass
class Saved:
    """What a forward pass keeps for the backward pass."""
    residual: torch.Tensor
    before: torch.Tensor
    y: torch.Tensor
    pre: torch.Tensor
    hidden: torch.Tensor
    z_in: torch.Tensor
    z_out: torch.Tensor


@dataclass
class Gradients:
    residual: torch.Tensor
    before: torch.Tensor
    weight: torch.Tensor
    post_weight: torch.Tensor
    gate: torch.Tensor
    adapters: tuple


class AdapterBlock:
    def __init__(self, w13, w2, weight, post_weight, gate, adapters, scale):
        """w13 [2F, H], w2 [H, F] bfloat16; weight and post_weight [H], gate [1, H] of the norms;
        adapters: a_in [L, R, H], b_in [L, 2F, R], a_out [L, R, F], b_out [L, H, R]; scale [L]."""
        self.w13, self.w2, self.weight, self.post_weight, self.gate = w13, w2, weight, post_weight, gate
        self.adapters, self.scale = adapters, scale

    def forward(self, residual: torch.Tensor, before: torch.Tensor, r: Requests, keep: bool = False):
        """residual, before (the output of the block before) [T, H] -> (this block's output, the
        residual stream, Saved or None)."""
        a_in, b_in, a_out, b_out = self.adapters
        y, stream = q.block_norm(residual, self.weight, block=before, block_weight=self.post_weight, gate=self.gate)
        part = q.lora_gemm(y, a_in, b_in, r.offsets, r.ids, scale=self.scale, return_z=keep)
        part, z_in = part if keep else (part, None)
        hidden = q.gated_gemm(self.w13, y, addend=part, return_pre=keep)
        hidden, pre = hidden if keep else (hidden, None)
        out = q.bf16_gemm(self.w2, hidden)
        done = q.lora_gemm(hidden, a_out, b_out, r.offsets, r.ids, scale=self.scale, base=out, out=out, return_z=keep)
        out, z_out = done if keep else (done, None)
        return out, stream, Saved(stream, before, y, pre, hidden, z_in, z_out) if keep else None

    def backward(self, grad_out: torch.Tensor, grad_stream: torch.Tensor, s: Saved, r: Requests) -> Gradients:
        a_in, b_in, a_out, b_out = self.adapters
        grad = q.bf16_gemm_grad_x(grad_out, self.w2)
        grad, ga_out, gb_out = q.lora_gemm_backward(grad_out, s.hidden, s.z_out, a_out, b_out, r.offsets, r.ids,
                                                    scale=self.scale, base=grad, grad_x=grad)
        grad_pre, grad_y, _ = q.gated_gemm_backward(grad, s.pre, self.w13, s.y, need_w=False)
        grad_y, ga_in, gb_in = q.lora_gemm_backward(grad_pre, s.y, s.z_in, a_in, b_in, r.offsets, r.ids,
                                                    scale=self.scale, base=grad_y, grad_x=grad_y)
        g = q.block_norm_backward(grad_y, grad_stream, s.residual, self.weight, block=s.before,
                                  block_weight=self.post_weight, gate=self.gate)
        return Gradients(g.residual, g.block, g.weight, g.block_weight, g.gate, (ga_in, gb_in, ga_out, gb_out))


def plain(block: AdapterBlock, residual, before, r: Requests, grad_out, grad_stream):
    """The same block in float32: (output, residual stream, gradients in Gradients' order)."""
    leaf = lambda t: t.float().requires_grad_(True)  # noqa: E731
    residual, before, weight, post, gate = map(leaf, (residual, before, block.weight, block.post_weight, block.gate))
    adapters = [leaf(t) for t in block.adapters]
    w13, w2 = block.w13.float(), block.w2.float()

    def norm(x, w):
        return x * torch.rsqrt((x * x).mean(1, keepdim=True) + 1e-6) * w

    def adapter(x, a, b):
        parts = []
        edges = r.offsets.tolist()
        for n, l in enumerate(r.ids.tolist()):
            rows = x[edges[n]:edges[n + 1]]
            parts.append(block.scale[l] * (rows @ a[l].t()) @ b[l].t() if l >= 0 else rows.new_zeros((len(rows), b.shape[1])))
        return torch.cat(parts)

    stream = residual + gate * norm(before, post)
    y = norm(stream, weight)
    g, u = (y @ w13.t() + adapter(y, adapters[0], adapters[1])).chunk(2, 1)
    hidden = torch.nn.functional.silu(g) * u
    out = hidden @ w2.t() + adapter(hidden, adapters[2], adapters[3])
    torch.autograd.backward((out, stream), (grad_out.float(), grad_stream.float()))
    return out.detach(), stream.detach(), [t.grad for t in (residual, before, weight, post, gate, *adapters)]


def make(counts, hidden: int = 512, inner: int = 704, adapters: int = 3, rank: int = 8, seed: int = 0):
    """A block, requests of `counts` rows, the last one without an adapter, and inputs and gradients."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g, device="cuda") * std + mean).bfloat16()

    weights = normal(2 * inner, hidden, std=hidden ** -0.5), normal(hidden, inner, std=inner ** -0.5)
    low = (normal(adapters, rank, hidden, std=hidden ** -0.5), normal(adapters, 2 * inner, rank, std=rank ** -0.5),
           normal(adapters, rank, inner, std=inner ** -0.5), normal(adapters, hidden, rank, std=rank ** -0.5))
    block = AdapterBlock(*weights, normal(hidden, std=0.2, mean=1.0), normal(hidden, std=0.2, mean=1.0), normal(1, hidden),
                         low, torch.rand(adapters, generator=g, device="cuda") + 0.5)
    rows = sum(counts)
    ids = [n % adapters for n in range(len(counts))]
    if len(counts) > 1:
        ids[-1] = -1
    requests = Requests(torch.tensor([sum(counts[:n]) for n in range(len(counts) + 1)], dtype=torch.int32, device="cuda"),
                        torch.tensor(ids, dtype=torch.int32, device="cuda"))
    return block, requests, [normal(rows, hidden) for _ in range(4)]


def run(counts, **sizes):
    """{name: relative distance to the plain block's} of the output, the stream and all gradients."""
    block, requests, (residual, before, grad_out, grad_stream) = make(counts, **sizes)
    out, stream, saved = block.forward(residual, before, requests, keep=True)
    g = block.backward(grad_out, grad_stream, saved, requests)
    want_out, want_stream, want = plain(block, residual, before, requests, grad_out, grad_stream)
    names = ["residual", "before", "weight", "post_weight", "gate", "a_in", "b_in", "a_out", "b_out"]
    got = [g.residual, g.before, g.weight, g.post_weight, g.gate, *g.adapters]

    def distance(a, b):
        return float((a.float() - b).norm() / b.norm())

    return {"out": distance(out, want_out), "stream": distance(stream, want_stream),
            **{n: distance(a, b) for n, a, b in zip(names, got, want)}}


if __name__ == "__main__":
    for counts in ([1], [1, 1, 1, 1], [40, 1, 70, 25], [900, 17, 1100, 300]):
        print(counts, {n: f"{d:.1e}" for n, d in run(counts).items()}, flush=True)
