"""The operators of a feed-forward block run together, as examples/adapter_block.py does: against its plain
float32 form, on streams of their own, and captured.

Distances: a pass rounds to bfloat16 the stream, the normed rows, the adapters' part, the hidden rows and the
output, each by at most 2^-8 of a value, and the backward pass the gradients of the hidden rows (twice), of both
factors, of the normed rows (twice) and its results; a relative distance, which roundings of independent
signs enter by their root mean square, is below the sum of half of them: 5 * 2^-9 for the output, 12 * 2^-9 for gradients."""

import os
import sys

import pytest
import torch

from gpu_util import show

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("counts,sizes", [([1], {}), ([1] * 6, {}), ([40, 1, 70, 25], {}), ([9, 33], dict(hidden=203, inner=131, rank=5)),
                                          ([300, 17, 500, 200], dict(hidden=1024, inner=1408, adapters=2, rank=16))])
def test_block(counts, sizes):
    import adapter_block
    show("adapter block", counts, sizes)
    for name, d in adapter_block.run(counts, **sizes).items():
        assert d <= (5 if name in ("out", "stream") else 12) * 2.0 ** -9, (name, d)


def flat(out, stream, g):
    return [out, stream, g.residual, g.before, g.weight, g.post_weight, g.gate, *g.adapters]


def step(made):
    block, requests, (residual, before, grad_out, grad_stream) = made
    out, stream, saved = block.forward(residual, before, requests, keep=True)
    return flat(out, stream, block.backward(grad_out, grad_stream, saved, requests))


def test_on_streams_of_their_own():
    """Two blocks' steps at once on two streams give what they give alone."""
    import adapter_block
    made = [adapter_block.make([40, 1, 70, 25], seed=1), adapter_block.make([130, 66, 3], hidden=768, inner=512, seed=2)]
    want = [[t.clone() for t in step(m)] for m in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    got = [None, None]
    for _ in range(4):
        for n, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[n] = step(made[n])
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("counts", [[1] * 5, [40, 1, 70, 25]])
def test_captured(counts):
    """Forward and backward pass in one graph, replayed on new inputs with eager work between."""
    import adapter_block
    made = adapter_block.make(counts, seed=3)
    others = [adapter_block.make(counts, seed=s)[2] for s in (4, 5, 6)]
    want = []
    for inputs in others:
        want.append([t.clone() for t in step((made[0], made[1], inputs))])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(made)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(made)
    for inputs, ref in zip(others * 2, want * 2):
        for to, new in zip(made[2], inputs):
            to.copy_(new)
        graph.replay()
        eager = step((made[0], made[1], inputs))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
        assert all(torch.equal(a, b) for a, b in zip(eager, ref))


def test_two_graphs_with_one_workspace_in_turn():
    """Two captured calls that were given the same workspace run one after the other."""
    import weight_quantized_linear_amd as q
    gen = torch.Generator(device="cuda").manual_seed(7)
    normal = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    off, ids = torch.tensor([0, 30, 64], dtype=torch.int32, device="cuda"), torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    calls = [(normal(64, 1024), normal(2, 16, 1024), normal(2, 256, 16)) for _ in range(2)]
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    want = [q.lora_gemm(*c, off, ids) for c in calls]
    graphs, got = [], []
    for c in calls:
        q.lora_gemm(*c, off, ids, workspace=ws)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(q.lora_gemm(*c, off, ids, workspace=ws))
    for _ in range(3):
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
