"""The expert layer of examples/expert_layer.py never waits for the GPU, so that
all of it can be captured in a graph.

Tolerance of a replay against the eager layer on the same inputs: all but two
steps give the same bits; y and the gradient of x add a token's two rows, and
the gradient of x a third term, in any order.  A sum of three 32-bit terms in
another order is off by at most 2 * 2^-24 of the terms' magnitudes: 1e-5 of the
result's 2-norm leaves room for terms 80 times the sum."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

TOKENS, WIDTH = 200, 192


def inputs(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    x = torch.randn((TOKENS, WIDTH), generator=gen, device="cuda").bfloat16()
    dy = torch.randn((TOKENS, WIDTH), generator=gen, device="cuda")
    masked = torch.rand((TOKENS, 6), generator=gen, device="cuda") < 0.3
    masked[::5] = True
    return x, dy, masked


def everything(layer, packed, x, dy, masked):
    y, grads = layer.step(x, dy, masked)
    return {"y": y, "forward": layer.forward(x, masked), "served": layer.serve(x, packed, masked), **grads}


def make():
    from expert_layer import ExpertLayer

    layer = ExpertLayer(width=WIDTH, hidden=320, experts=6, choices=2, seed=3)
    return layer, layer.pack()


def test_no_step_waits_for_the_gpu():
    layer, packed = make()
    args = inputs(1)
    want = everything(layer, packed, *args)
    torch.cuda.synchronize()
    torch.cuda.set_sync_debug_mode("error")
    try:
        everything(layer, packed, *args)
    finally:
        torch.cuda.set_sync_debug_mode("default")
    assert all(v.isfinite().all() for v in want.values())


def test_captured_layer():
    layer, packed = make()
    static = inputs(2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                        # plans and workspaces of this stream
        everything(layer, packed, *static)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        captured = everything(layer, packed, *static)
    for seed in range(3, 7):
        fresh = inputs(seed)
        for s, f in zip(static, fresh):
            s.copy_(f)
        graph.replay()
        torch.cuda.synchronize()
        want = everything(layer, packed, *fresh)
        torch.cuda.synchronize()
        for name, v in want.items():
            off = (captured[name].double() - v.double()).norm() / v.double().norm()
            assert off <= 1e-5, f"{name} of the replay on seed {seed}: {off:.2e}"
