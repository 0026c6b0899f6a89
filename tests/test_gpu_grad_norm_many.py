"""Clipping of lists that take many launches: what each costs does not grow with
their number."""
from __future__ import annotations

import math

import pytest
import torch

import layer_refs as R
from gpu_support import say
from shared_memory_tiled_amd import binding

pytestmark = pytest.mark.gpu


def captured(call, calls=3):
    """(what the last replay left, microseconds of a call: the least of five replays)."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(calls):
            result = call()
    times = []
    for _ in range(5):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        graph.replay()
        end.record()
        torch.cuda.synchronize()
        times.append(start.elapsed_time(end) * 1e3 / calls)
    return result, min(times)


def test_no_slower_than_its_two_calls():
    """5000 tensors of 16 chunks: 40 launches of 2048 partial sums each."""
    count, size = 5000, 1 << 16
    say(f"clip {count} x {size}")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    grads = [torch.randn(size, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(count)]
    out, other = [torch.empty_like(g) for g in grads], [torch.empty_like(g) for g in grads]
    n1, both = captured(lambda: binding.clip_grad_norm(grads, 0.5, out=out))

    def apart():
        norm = binding.grad_norm(grads)
        binding.clip_grads(grads, norm, 0.5, out=other)
        return norm

    n2, two = captured(apart)
    want = math.sqrt(sum(g.double().square().sum().item() for g in grads))
    assert abs(n1.item() - want) <= want * (2.0 ** -24 + 1e-9) and torch.equal(n1, n2)
    assert all(torch.equal(a, b) for a, b in zip(out, other))
    assert both <= 2 * two, (both, two)


@pytest.mark.parametrize("count", [127, 128, 129, 256, 257, 400])
def test_counts_about_a_launch(count):
    """Tensors that end with a launch, or begin another; empty ones after the last."""
    grads = [torch.full((50 + i % 7,), 0.5 + i % 3, device="cuda") for i in range(count)] + [torch.empty(0, device="cuda")] * 3
    want = math.sqrt(sum(g.double().square().sum().item() for g in grads))
    out = [torch.full_like(g, 7.0) for g in grads]
    norm = binding.clip_grad_norm(grads, 1.0, out=out)
    assert abs(norm.item() - want) <= want * (2.0 ** -24 + 1e-9)
    for g, o in zip(grads, out):
        ref = g.double() / (want + 1e-6)
        R.within(o, ref, 4.2 * R.U * ref, "clipped")
