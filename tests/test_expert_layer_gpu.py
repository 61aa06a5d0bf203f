"""The operators run together as an expert layer uses them (examples/
expert_layer.py), against the same layer in 64 bits with automatic
differentiation.

Tolerance: every stage of the layer rounds to bfloat16, each rounding 2^-8 of
a value; a gradient passes at most 8 of them in a row, and errors of a sum's
terms add at most linearly: 8 * 2^-8 in the 2-norm.  4-bit operands are off by
up to a quarter of a value (half the step between 4 and 6 over 4 is a quarter);
two products with both operands in 4 bits: below 1 in the 2-norm, and not 0."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("tokens,masking", [(1, False), (7, True), (300, True), (700, False)])
def test_expert_layer(tokens, masking):
    from expert_layer import ExpertLayer, gelu

    layer = ExpertLayer(width=192, hidden=320, experts=6, choices=2, seed=tokens)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(tokens + 1)
    x = torch.randn((tokens, 192), generator=gen, device="cuda").bfloat16()
    dy = torch.randn((tokens, 192), generator=gen, device="cuda")
    masked = None
    if masking:
        masked = torch.rand((tokens, 6), generator=gen, device="cuda") < 0.3
        masked[::5] = True
    y, grads = layer.step(x, dy, masked)

    leaf = {"x": x.double(), "router": layer.router.double(), "w1": layer.w1.double(), "b1": layer.b1.double(),
            "w2": layer.w2.double()}
    leaf = {k: v.cpu().requires_grad_() for k, v in leaf.items()}
    logits = leaf["x"] @ leaf["router"]
    if masked is not None:
        logits = logits.masked_fill(masked.cpu(), float("-inf"))
    # The library's own choice of experts, so that a near tie does not decide.
    experts = layer._dispatch(x, masked)[1].experts.long().cpu()
    out = torch.zeros((tokens, 192), dtype=torch.float64)
    rows = []
    for t in range(tokens):
        e = experts[t][experts[t] >= 0]
        if len(e) == 0:
            rows.append(out[t])
            continue
        w = torch.softmax(logits[t][e], 0)
        rows.append(sum(w[i] * (gelu(leaf["x"][t] @ leaf["w1"][n] + leaf["b1"][n]) @ leaf["w2"][n])
                        for i, n in enumerate(e.tolist())))
    ref = torch.stack(rows)
    (ref * dy.double().cpu()).sum().backward()

    def off(a, b):
        return ((a.double().cpu() - b).norm() / b.norm().clamp(min=1e-30)).item()

    assert off(y, ref.detach()) <= 8 * 2 ** -8
    for name, got in grads.items():
        want = leaf[name].grad
        assert off(got, want) <= 8 * 2 ** -8, name
    assert off(layer.forward(x, masked), ref.detach()) <= 8 * 2 ** -8
    served = layer.serve(x, layer.pack(), masked)
    assert 0 < off(served, ref.detach()) < 1
    if masked is not None:
        assert (served[::5] == 0).all() and (y[::5] == 0).all()
