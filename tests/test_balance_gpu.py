"""Balanced routing on the GPU against a plain implementation in 64 bits, token
by token: which experts are chosen exactly, weights and gradients within their
roundings.

Tolerances.  Weights are computed in 64 bits and rounded once to 32: 2^-24 of the
value.  A gradient is w (g - dot / scale) / (1 + e^x) in 32 bits: dot sums up to
`choices` products that are rounded once each (sum and product: 2 choices
roundings of their magnitudes), w carries one rounding, and the difference, the
division by scale, the exponential (two units at most, 4 roundings), the sum, the
division and the product come to 9 more; softmax over all experts sums up to 64
terms a lane and 4 between lanes, each exponential off by 4: 80.  So
(2 choices + 90) 2^-24 w (|g| + sum w |g| / scale) bounds each term, plus half a
step of the logits' type."""
import math

import pytest
import torch

import dense_gemm_optimisation_fp32_amd as g

pytestmark = pytest.mark.gpu
INF = float("inf")


def scores_of(row, kind):
    if kind == "sigmoid":
        return [1.0 / (1.0 + math.exp(-x)) if x > -700 else 0.0 for x in row]
    live = [x for x in row if x > -INF]
    if not live:
        return [0.0] * len(row)
    top = max(live)
    p = [math.exp(x - top) if x > -INF else 0.0 for x in row]
    total = math.fsum(p)
    return [v / total for v in p]


def reference(logits, choices, bias, kind, sets, kept, normalize, scale):
    """Per token: chosen experts and their weights."""
    experts, weights, scores = [], [], []
    for row in logits:
        row = [-INF if x != x else x for x in row]
        s = scores_of(row, kind)
        key = [-INF if x == -INF or b != b else v + b for x, v, b in zip(row, s, bias)]
        size = len(row) // sets
        values = []
        for i in range(sets):
            two = sorted((k for k in key[i * size:(i + 1) * size] if k > -INF), reverse=True)[:2]
            values.append(sum(two) if two else -INF)
        ranked = sorted(range(sets), key=lambda i: (-values[i], i))[:kept]
        allowed = [e for e in range(len(row)) if e // size in ranked and key[e] > -INF]
        pick = sorted(allowed, key=lambda e: (-key[e], e))[:choices]
        total = math.fsum(s[e] for e in pick) if normalize else 1.0
        weights.append([scale * s[e] / total if total > 0 else 0.0 for e in pick] + [0.0] * (choices - len(pick)))
        experts.append(pick + [-1] * (choices - len(pick)))
        scores.append(s)
    return experts, weights, scores


def gradient(row, s, pick, w, grad, kind, normalize, scale):
    """The logits' gradient of one token, and the magnitudes that its roundings go by."""
    d, size = [0.0] * len(row), [0.0] * len(row)
    live = [j for j, e in enumerate(pick) if e >= 0]
    dot = math.fsum(w[j] * grad[j] for j in live)
    much = math.fsum(abs(w[j] * grad[j]) for j in live)
    for j in live:
        e = pick[j]
        slope = 1.0 / (1.0 + math.exp(row[e])) if kind == "sigmoid" else 1.0
        d[e] += w[j] * (grad[j] - (dot / scale if normalize else 0.0)) * slope
        size[e] += w[j] * (abs(grad[j]) + (much / scale if normalize else 0.0)) * slope
    if kind == "softmax" and not normalize:
        for e in range(len(row)):
            d[e] -= s[e] * dot
            size[e] += s[e] * much
    return d, size


def check(logits, choices, bias=None, kind="sigmoid", sets=1, kept=1, normalize=True, scale=1.0, seed=0):
    dtype, (tokens, groups) = logits.dtype, logits.shape
    r = g.route_balanced(logits, choices, bias=bias, scores=kind, sets=sets, kept_sets=kept, normalize=normalize, scale=scale)
    rows = logits.double().cpu().tolist()
    b = [0.0] * groups if bias is None else bias.double().cpu().tolist()
    experts, weights, scores = reference(rows, choices, b, kind, sets, kept, normalize, scale)
    assert r.experts.cpu().tolist() == experts
    want = torch.tensor(weights, dtype=torch.float64).reshape(tokens, choices)
    off = (r.weights.double().cpu() - want).abs()
    assert (off <= want * 2.0 ** -24 * 1.001 + 1e-300).all(), off.max().item()
    slots = sorted((e, t * choices + j) for t, pick in enumerate(experts) for j, e in enumerate(pick) if e >= 0)
    order = [s for _, s in slots]
    assert r.order.cpu().tolist() == order + [-1] * (tokens * choices - len(order))
    assert r.offsets.cpu().tolist() == [sum(1 for e, _ in slots if e < i) for i in range(groups + 1)]

    gen = torch.Generator().manual_seed(seed)
    grad = torch.randn((tokens, choices), generator=gen)
    got = g.route_balanced_grad(logits, r, grad.cuda())
    assert got.dtype == dtype and got.shape == logits.shape
    got = got.double().cpu()
    for t in range(tokens):
        row = [-INF if x != x else x for x in rows[t]]
        d, size = gradient(row, scores[t], experts[t], weights[t], grad[t].tolist(), kind, normalize, scale)
        d, size = torch.tensor(d, dtype=torch.float64), torch.tensor(size, dtype=torch.float64)
        room = (2 * choices + 90) * 2.0 ** -24 * size + torch.finfo(dtype).eps / 2 * d.abs() + 1e-38
        assert ((got[t] - d).abs() <= room * 1.001).all(), (t, (got[t] - d).abs().max())
    return r


def normal(tokens, groups, dtype, seed, scale=1.5):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((tokens, groups), generator=gen, device="cuda") * scale).to(dtype)


SHAPES = [  # tokens, groups, choices, sets, kept
    (1, 1, 1, 1, 1), (1, 2, 2, 2, 2), (3, 7, 7, 1, 1), (16, 64, 4, 8, 4), (17, 60, 6, 6, 3), (5, 16, 3, 16, 4), (9, 33, 5, 3, 2),
    (129, 40, 8, 5, 3), (128, 256, 8, 8, 4), (300, 255, 8, 5, 2), (20, 384, 8, 8, 4), (7, 340, 8, 17, 9), (6, 64, 8, 64, 11),
    (4, 130, 32, 2, 1), (140, 513, 8, 3, 2), (5, 1024, 32, 1, 1), (5, 1020, 8, 3, 2), (3, 1024, 9, 64, 16), (131, 512, 6, 1, 1),
    (4, 1000, 20, 40, 30),
]


@pytest.mark.parametrize("kind,normalize", [("sigmoid", True), ("sigmoid", False), ("softmax", True), ("softmax", False)])
@pytest.mark.parametrize("tokens,groups,choices,sets,kept", SHAPES)
def test_routes(tokens, groups, choices, sets, kept, kind, normalize):
    dtype = torch.float32 if (tokens + groups) % 2 else torch.bfloat16
    logits = normal(tokens, groups, dtype, tokens * 7 + groups)
    bias = normal(1, groups, torch.float32, groups, 0.1 if kind == "sigmoid" else 0.3 / groups)[0]
    check(logits, choices, bias, kind, sets, kept, normalize, 2.5)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masked_rows_and_sets(kind, dtype):
    """Padded tokens, sets with one expert or none left, experts masked for all."""
    logits = normal(150, 48, dtype, 3)
    logits[::7] = -INF                        # no expert
    logits[1::7, 2:] = -INF                   # two of one set
    logits[2::7, 1:] = -INF                   # one
    logits[3::7, :40] = -INF                  # one set
    logits[4::7, torch.arange(48) % 8 != 3] = -INF        # one of each set
    logits[5::7, 5] = float("nan")
    bias = normal(1, 48, torch.float32, 4, 0.1)[0]
    bias[9] = -INF
    for choices, sets, kept in ((4, 6, 3), (8, 1, 1), (3, 6, 6), (6, 3, 1)):
        check(logits, choices, bias, kind, sets, kept)


@pytest.mark.parametrize("sets,kept", [(1, 1), (8, 3), (6, 2)])
def test_ties_go_to_the_lowest(sets, kept):
    check(torch.zeros((40, 48), device="cuda"), 6, None, "sigmoid", sets, kept)
    # bfloat16 logits of few values.
    logits = (normal(200, 48, torch.float32, 9) * 2).round().bfloat16() / 2
    check(logits, 6, None, "sigmoid", sets, kept)
    check(logits, 6, torch.zeros(48, device="cuda"), "softmax", sets, kept)


@pytest.mark.parametrize("groups", [16, 64, 120, 256, 384, 1024])
@pytest.mark.parametrize("choices", [1, 7, 8, 9, 16])
def test_neighbours_hold_all_choices(groups, choices):
    """Every choice from neighbouring experts, from either end, and keys of both signs."""
    up = torch.linspace(-3.0, 3.0, groups).repeat(6, 1)
    up[1] = up[1].flip(0)
    up[2, : groups // 2] = up[2, : groups // 2].flip(0)
    up[3:] = up[3:].roll(groups // 3, 1)
    bias = torch.full((groups,), -0.5)
    for kind in ("sigmoid", "softmax"):
        for dtype in (torch.float32, torch.bfloat16):       # (in 16 bits many are equal)
            check(up.to(dtype).cuda(), choices, bias.cuda(), kind)


def test_choice_goes_by_64_bits():
    """Keys that 32 bits cannot tell apart: sigmoids of neighbouring 32-bit logits
    near 9, a bias that all but makes up for their difference."""
    x = torch.full((64, 32), 9.0, device="cuda")
    step = torch.arange(32, device="cuda", dtype=torch.float32) * 2.0 ** -20
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = x + step[torch.rand((64, 32), generator=gen, device="cuda").argsort(1)]
    check(x, 8, None, "sigmoid", 4, 2)


def test_far_logits_and_infinities():
    x = normal(64, 32, torch.float32, 8) * 60
    x[3, 4] = INF                             # a sigmoid of one
    check(x, 4, None, "sigmoid", 4, 2, scale=0.75)
    y = torch.full((3, 8), -1e30, device="cuda")          # sigmoids of zero: weights are 0
    r = g.route_balanced(y, 2)
    assert (r.weights == 0).all() and r.experts.tolist() == [[0, 1]] * 3
    assert (g.route_balanced_grad(y, r, torch.ones((3, 2), device="cuda")) == 0).all()


def test_strided_logits_and_no_tokens():
    wide = normal(50, 100, torch.bfloat16, 11)
    check(wide[::2, 3:67], 5, None, "softmax", 4, 2, False, 1.5)
    r = g.route_balanced(torch.empty((0, 12), device="cuda"), 3, sets=3, kept_sets=2)
    assert r.offsets.tolist() == [0] * 13 and r.weights.shape == (0, 3) and r.order.numel() == 0
    assert g.route_balanced_grad(torch.empty((0, 12), device="cuda"), r, torch.empty((0, 3), device="cuda")).shape == (0, 12)


def test_without_sets_and_bias_it_is_route():
    """Softmax scores, renormalised, without bias or sets choose as route does."""
    x = normal(500, 64, torch.float32, 13)
    a, b = g.route(x, 6), g.route_balanced(x, 6, scores="softmax")
    assert torch.equal(a.experts, b.experts) and torch.equal(a.order, b.order) and torch.equal(a.offsets, b.offsets)
    assert (a.weights - b.weights).abs().max() <= 2.0 ** -20


@pytest.mark.parametrize("kind,normalize", [("sigmoid", True), ("sigmoid", False), ("softmax", True), ("softmax", False)])
def test_gradient_against_differences(kind, normalize):
    """d (sum w g) by central differences of the 64-bit weights: the step's error is h^2 times a
    third derivative (below 10 of these smooth functions times scale): h = 1e-4."""
    x = normal(6, 24, torch.float32, 21)
    grad = torch.randn((6, 5), generator=torch.Generator().manual_seed(2))
    r = g.route_balanced(x, 5, scores=kind, sets=4, kept_sets=3, normalize=normalize, scale=1.5)
    got = g.route_balanced_grad(x, r, grad.cuda()).cpu()
    rows, pick, h = x.double().cpu().tolist(), r.experts.tolist(), 1e-4
    for t in range(6):
        for e in range(24):
            f = []
            for sign in (1, -1):
                row = list(rows[t])
                row[e] += sign * h
                s = scores_of(row, kind)
                total = math.fsum(s[i] for i in pick[t]) if normalize else 1.0
                f.append(math.fsum(1.5 * s[i] / total * w for i, w in zip(pick[t], grad[t].tolist())))
            assert abs((f[0] - f[1]) / (2 * h) - got[t, e].item()) <= 1e-6


def test_many_tokens_keep_their_order():
    """Whole workgroups and a part of one: every slot once, sorted."""
    x = normal(20000, 96, torch.bfloat16, 31)
    r = g.route_balanced(x, 6, sets=8, kept_sets=4, bias=normal(1, 96, torch.float32, 32, 0.1)[0])
    flat = r.experts.reshape(-1).long()
    assert torch.equal(torch.sort(flat, stable=True)[1].int(), r.order)
    assert torch.equal(torch.bincount(flat, minlength=96).cumsum(0).int(), r.offsets[1:])


def test_captured_and_replayed():
    x, bias = normal(700, 64, torch.float32, 41), normal(1, 64, torch.float32, 42, 0.1)[0]
    grad = torch.randn((700, 4), device="cuda")

    def once():
        r = g.route_balanced(x, 4, bias=bias, sets=8, kept_sets=4)
        return r.weights, r.experts, r.offsets, r.order, g.route_balanced_grad(x, r, grad)

    once()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = once()
    for seed in range(3):
        x.copy_(normal(700, 64, torch.float32, 50 + seed))
        bias.copy_(normal(1, 64, torch.float32, 60 + seed, 0.1)[0])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, once()))


def test_two_streams_at_once():
    x = [normal(5000, 128, torch.float32, s) for s in (71, 72)]
    want = [g.route_balanced(v, 8, sets=8, kept_sets=4) for v in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in x]
    for _ in range(3):
        got = []
        for v, s in zip(x, streams):
            with torch.cuda.stream(s):
                got.append(g.route_balanced(v, 8, sets=8, kept_sets=4))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a.order, b.order) and torch.equal(a.weights, b.weights)


def test_refusals():
    x = normal(5, 12, torch.float32, 1)
    for bad in (dict(sets=5), dict(sets=0), dict(sets=3, kept_sets=4), dict(sets=3, kept_sets=0), dict(scale=0.0),
                dict(scale=float("nan")), dict(bias=torch.zeros(11, device="cuda")), dict(bias=torch.zeros(12)),
                dict(bias=torch.zeros(12, device="cuda").double()), dict(bias=torch.zeros(24, device="cuda")[::2])):
        with pytest.raises(ValueError):
            g.route_balanced(x, 2, **bad)
    for choices in (0, 13):
        with pytest.raises(ValueError):
            g.route_balanced(x, choices)
    with pytest.raises(ValueError):
        g.route_balanced(x, 5, sets=3, kept_sets=1)           # four experts are left
    with pytest.raises(g.GemmF32Error):
        g.route_balanced(normal(5, 64, torch.float32, 1), 33)
    with pytest.raises(ValueError):
        g.route_balanced(x.t(), 2)
    r = g.route_balanced(x, 2)
    for grad in (torch.zeros((5, 3), device="cuda"), torch.zeros((5, 2)), torch.zeros((5, 2), device="cuda").double()):
        with pytest.raises(ValueError):
            g.route_balanced_grad(x, r, grad)
    with pytest.raises(ValueError):
        g.route_balanced_grad(x[:4], r, torch.zeros((5, 2), device="cuda"))


def test_experts_outside_the_range_are_left_out():
    """A gradient of experts that there are not (a list that the caller changed) stays inside."""
    x = normal(40, 12, torch.float32, 1)
    r = g.route_balanced(x, 3)
    r.experts[::2, 1] = 12
    r.experts[1::2, 0] = -7
    wide = torch.full((42, 12), 3.0, device="cuda")
    wide[1:41] = g.route_balanced_grad(x, r, torch.ones((40, 3), device="cuda"))
    assert wide.isfinite().all() and (wide[0] == 3).all() and (wide[41] == 3).all()
