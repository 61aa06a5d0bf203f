"""Balanced routing, 8-bit products and orthogonalised updates together, as a layer
uses them (examples/balanced_layer.py), against the same layer in 64 bits with
automatic differentiation, and captured in a graph.

Tolerance: every stage rounds to bfloat16, 2^-8 of a value each; a gradient passes at
most 8 of them in a row: 8 * 2^-8 in the 2-norm.  8-bit operands are off by half a step,
1/254 of a row's largest value, whose size is at most 6 deviations of the normal rows
here: 6 / 254 / sqrt(3) of the 2-norm an operand, two operands in each of two products:
4 * 0.014 = 0.055, and the bfloat16 roundings.  An update is orthogonal up to the steps'
range of singular values and bfloat16: compared with the same steps of the same
gradient in 64 bits, 2^-8 for the update, one for the subtraction, 5 * 2^-11 inside."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
WIDTH, HIDDEN, EXPERTS = 192, 320, 12


def make(seed):
    from balanced_layer import BalancedLayer

    layer = BalancedLayer(width=WIDTH, hidden=HIDDEN, experts=EXPERTS, choices=3, sets=4, seed=seed)
    layer.balance += 0.1 * torch.randn(EXPERTS, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")
    return layer


def inputs(tokens, masking, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((tokens, WIDTH), generator=gen, device="cuda").bfloat16()
    dy = torch.randn((tokens, WIDTH), generator=gen, device="cuda")
    masked = None
    if masking:
        masked = torch.rand((tokens, EXPERTS), generator=gen, device="cuda") < 0.3
        masked[::5] = True
    return x, dy, masked


def off(a, b):
    return ((a.double().cpu() - b).norm() / b.norm().clamp(min=1e-30)).item()


@pytest.mark.parametrize("tokens,masking", [(1, False), (9, True), (300, True), (700, False)])
def test_layer_against_64_bits(tokens, masking):
    from expert_layer import gelu

    layer = make(tokens)
    x, dy, masked = inputs(tokens, masking, tokens + 1)
    y, grads = layer.step(x, dy, masked)
    leaf = {k: v.double().cpu().requires_grad_() for k, v in
            {"x": x, "router": layer.router, "w1": layer.w1, "b1": layer.b1, "w2": layer.w2}.items()}
    score = torch.sigmoid(leaf["x"] @ leaf["router"])
    experts = layer._dispatch(x, masked)[1].experts.long().cpu()
    rows = []
    for t in range(tokens):
        e = experts[t][experts[t] >= 0]
        if len(e) == 0:
            rows.append(torch.zeros(WIDTH, dtype=torch.float64))
            continue
        w = 2.5 * score[t][e] / score[t][e].sum()
        rows.append(sum(w[i] * (gelu(leaf["x"][t] @ leaf["w1"][n] + leaf["b1"][n]) @ leaf["w2"][n]) for i, n in enumerate(e.tolist())))
    ref = torch.stack(rows)
    (ref * dy.double().cpu()).sum().backward()
    assert off(y, ref.detach()) <= 8 * 2 ** -8
    for name, got in grads.items():
        assert off(got, leaf[name].grad) <= 8 * 2 ** -8, name
    served = layer.serve8(x, layer.pack8(), masked)
    assert off(served, ref.detach()) <= 0.055 + 4 * 2 ** -8
    if masked is not None:
        assert (served[::5] == 0).all() and (y[::5] == 0).all()


def test_update_against_64_bits():
    layer = make(5)
    x, dy, masked = inputs(400, True, 6)
    before = {k: getattr(layer, k).double().cpu() for k in ("w1", "w2", "balance")}
    loads = layer._dispatch(x, masked)[1].offsets.diff().double().cpu()
    _, grads = layer.update(x, dy, masked)
    for name in ("w1", "w2"):
        v = grads[name].double().cpu()
        v = v / v.flatten(1).norm(dim=1).clamp(min=1e-300).view(-1, 1, 1)
        for _ in range(5):
            s = v @ v.transpose(1, 2)
            v = 3.4445 * v + (-4.7750 * s + 2.0315 * s @ s) @ v
        scale = 0.02 * max(1.0, v.shape[2] / v.shape[1]) ** 0.5
        want = before[name] - scale * v
        got = getattr(layer, name).double().cpu()
        room = (2 ** -8 + 5 * 2 ** -11) * (scale * v).norm() + 2 ** -8 * want.norm()
        assert (got - want).norm() <= room, name
    want = before["balance"] + 0.01 * torch.sign(loads.mean() - loads)
    assert (layer.balance.double().cpu() - want).abs().max() <= 2.0 ** -23


def test_whole_layer_captured_and_replayed():
    """A step, the updates of its gradients and 8-bit serving in one graph, replayed on new
    inputs with eager work between; sums of a token's rows add in any order: 1e-5."""
    from balanced_layer import g

    layer = make(3)
    packed = layer.pack8()
    static = inputs(200, True, 2)

    def everything(x, dy, masked):
        y, grads = layer.step(x, dy, masked)
        return {"y": y, "served": layer.serve8(x, packed, masked), "u1": g.orthogonalize(grads["w1"]), "u2": g.orthogonalize(grads["w2"]),
                "x": grads["x"]}

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        everything(*static)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        captured = everything(*static)
    for seed in range(3, 7):
        fresh = inputs(200, True, seed)
        for s, f in zip(static, fresh):
            s.copy_(f)
        graph.replay()
        torch.cuda.synchronize()
        want = everything(*fresh)
        torch.cuda.synchronize()
        for name, v in want.items():
            assert (captured[name].double() - v.double()).norm() <= 1e-5 * v.double().norm(), (name, seed)
