"""The expert-layer and 4-bit operators, as they are measured.

Four operators, each in two forms: a plain one (elementary torch operations in
32 bits, rounded once at the end) and, where ``own`` is true, the calls that a
user makes of this library.

grouped   C_e = act(A_e . B_e + bias_e) for the experts e of an expert layer.
          A's rows are sorted by expert; offsets[e] .. offsets[e + 1] are e's
          rows.  A training step adds dA_e = G_e . B_e^T and dB_e = A_e^T . G_e.
pack      microscaled 4-bit floating point: blocks of 32 values along k share
          a power of two, each value is one of 0, .5, 1, 1.5, 2, 3, 4, 6 with
          a sign.  Quantised, and back to the values that the codes stand for.
mx4       Y = Q(X) . W^T with W held in 4 bits and X quantised on the way;
          with groups > 0 each expert has its own W.
route     softmax over the experts' logits, the k largest, and the order of
          the chosen (token, choice) slots sorted by expert; a training step
          adds the logits' gradient.

A 4-bit matrix of r rows and k columns is held as codes (r, kp / 2) and scales
(kp / 128, r, 4), kp = k rounded up to 128: two codes a byte, the even column
in the low half, and a byte 127 + e for a block's scale 2^e.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --- cases -------------------------------------------------------------------

def _grouped(name, m, n, k, groups, dtype, layout, step, bias, act, skew):
    return dict(name=name, op="grouped", m=m, n=n, k=k, groups=groups, dtype=dtype, layout=layout, step=step,
                bias=bias, act=act, skew=skew)


def _mx4(name, m, n, k, groups, dtype, skew):
    return dict(name=name, op="mx4", m=m, n=n, k=k, groups=groups, dtype=dtype, skew=skew)


def _pack(name, rows, k, dtype, along):
    return dict(name=name, op="pack", rows=rows, k=k, dtype=dtype, along=along)


def _route(name, tokens, groups, choices, dtype, normalize, masked, step):
    return dict(name=name, op="route", tokens=tokens, groups=groups, choices=choices, dtype=dtype,
                normalize=normalize, masked=masked, step=step)


def listed():
    return [
        # One token's two experts of eight in 32 bits: the smallest call, where latency counts.
        _grouped("grouped_token_f32", 2, 4096, 1024, 8, "f32", "col", False, False, "none", 0.0),
        # Eight sequences that decode together, two experts each: the weights' bytes count.
        _grouped("grouped_decode_bf16", 16, 14336, 4096, 8, "bf16", "col", False, False, "none", 0.3),
        # Prompts through the first product of an expert layer, with its bias and activation.
        _grouped("grouped_prompt_bf16", 16384, 14336, 4096, 8, "bf16", "col", False, True, "gelu", 0.3),
        # A training step of an expert layer's product: forward and both gradients, uneven experts.
        _grouped("grouped_step_bf16", 8192, 4096, 2048, 16, "bf16", "row", True, False, "none", 0.5),
        # The same in 32 bits on sizes that fit no tile.
        _grouped("grouped_step_f32", 5003, 1027, 2049, 16, "f32", "row", True, True, "none", 0.5),
        # An activation that goes to 4 bits between two small layers, blocks along the other axis (for a gradient).
        _pack("pack_turned_f32", 1000, 1025, "f32", "columns"),
        # A linear layer's weights packed once after loading.
        _pack("pack_weights_bf16", 14336, 4096, "bf16", "rows"),
        # Four sequences that decode through a linear layer with 4-bit weights.
        _mx4("mx4_decode_bf16", 4, 14336, 4096, 0, "bf16", 0.0),
        # A prompt through the same layer.
        _mx4("mx4_prompt_bf16", 8192, 14336, 4096, 0, "bf16", 0.0),
        # A short prompt through 32 experts with 4-bit weights, results in 32 bits.
        _mx4("mx4_experts_f32", 2049, 4096, 2048, 32, "f32", 0.5),
        # The router of one decoding step.
        _route("route_decode_f32", 16, 64, 4, "f32", True, 0.0, False),
        # The router of a training step with padded tokens and experts that a token may not use.
        _route("route_step_bf16", 32768, 128, 8, "bf16", True, 0.25, True),
    ]


def _between(rng, low, high):
    """A whole number of [low, high], even over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _size(rng, low, high):
    """As _between; two of three times a multiple of 64 where that fits, as layers' sizes are."""
    v = _between(rng, low, high)
    return max(64, v // 64 * 64) if v >= 64 and rng.random() < 0.67 else v


def draw(rng):
    op = rng.choice(("grouped", "grouped", "mx4", "mx4", "pack", "route"))
    dtype = rng.choice(("f32", "bf16"))
    if op == "grouped":
        groups = _between(rng, 1, 64)
        n, k = _size(rng, 64, 8192), _size(rng, 64, 8192)
        while groups * n * k > 8 * 14336 * 4096:
            groups = max(1, groups // 2)
        step = rng.random() < 0.5
        m = _between(rng, 1, min(16384, max(1, int(8e11 / (3 if step else 1) / (2 * n * k)))))
        return _drop_name(_grouped("", m, n, k, groups, dtype, rng.choice(("row", "col")), step,
                                   rng.random() < 0.5, "none" if step else rng.choice(("none", "relu", "gelu")),
                                   rng.choice((0.0, 0.3, 0.5))))
    if op == "mx4":
        groups = rng.choice((0, 0, _between(rng, 1, 64)))
        n, k = _size(rng, 64, 14336), _size(rng, 64, 8192)
        while max(1, groups) * n * k > 8 * 4096 * 4096:
            groups, n = groups // 2, (n if groups > 1 else n // 2)
        m = _between(rng, 1, min(8192, max(1, int(9e11 / (2 * n * k)))))
        return _drop_name(_mx4("", m, n, k, groups, dtype, rng.choice((0.0, 0.3, 0.5)) if groups else 0.0))
    if op == "pack":
        return _drop_name(_pack("", _size(rng, 1, 8192), _size(rng, 32, 7168), dtype, rng.choice(("rows", "columns"))))
    groups = _between(rng, 2, 256)
    return _drop_name(_route("", _between(rng, 1, 32768), groups, rng.randint(1, min(8, groups)), dtype,
                             rng.random() < 0.7, rng.choice((0.0, 0.25)), rng.random() < 0.5))


def _drop_name(case):
    return {key: v for key, v in case.items() if key != "name"}


# --- inputs ------------------------------------------------------------------

def _group_sizes(case, seed):
    """How many of the m rows each expert gets: uneven by `skew`, some experts without any."""
    rng = random.Random(seed * 7919 + 17)
    weights = [math.exp(case["skew"] * rng.gauss(0.0, 1.0)) for _ in range(case["groups"])]
    sizes = [0] * case["groups"]
    for e in rng.choices(range(case["groups"]), weights, k=case["m"]):
        sizes[e] += 1
    return sizes


def _generator(seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed))
    return gen


def _normal(gen, shape, scale, dtype):
    return (torch.randn(shape, generator=gen, device=DEVICE) * scale).to(TYPES[dtype])


def _offsets(sizes):
    ends = [0]
    for s in sizes:
        ends.append(ends[-1] + s)
    return torch.tensor(ends, dtype=torch.int32, device=DEVICE)


def prepare(case, seed):
    gen = _generator(seed)
    s = {"case": case}
    if case["op"] == "route":
        t, e = case["tokens"], case["groups"]
        logits = _normal(gen, (t, e), 1.5, case["dtype"])
        if case["masked"]:
            # Experts that a token may not use, and padded tokens, which use none.
            off = torch.rand((t, e), generator=gen, device=DEVICE) < case["masked"]
            off |= torch.rand((t, 1), generator=gen, device=DEVICE) < 0.05
            logits = logits.masked_fill(off, float("-inf"))
        s["logits"] = logits
        s["grad"] = _normal(gen, (t, case["choices"]), 1.0, "f32") if case["step"] else None
        return s
    if case["op"] == "pack":
        shape = (case["rows"], case["k"]) if case["along"] == "rows" else (case["k"], case["rows"])
        x = _normal(gen, shape, 1.0, "f32")
        # Rows and columns of different magnitude, as weights and activations have them.
        x *= torch.exp(torch.randn((shape[0], 1), generator=gen, device=DEVICE))
        s["x"] = x.to(TYPES[case["dtype"]])
        return s
    m, n, k, e = case["m"], case["n"], case["k"], case["groups"]
    s["a"] = _normal(gen, (m, k), 1.0, case["dtype"])
    s["offsets"], s["longest"] = None, m
    if e:
        sizes = _group_sizes(case, seed)
        s["offsets"], s["longest"] = _offsets(sizes), max(1, max(sizes))
    if case["op"] == "mx4":
        codes, scales = [], []
        for _ in range(max(1, e)):
            c, f = _encode(_normal(gen, (n, k), k ** -0.5, "f32"))
            codes.append(c)
            scales.append(f)
        s["codes"] = torch.stack(codes) if e else codes[0]
        s["scales"] = torch.stack(scales) if e else scales[0]
        return s
    # A linear layer's weights: (e, k, n), or held as (e, n, k) and seen transposed.
    s["b"] = torch.empty((e, k, n) if case["layout"] == "row" else (e, n, k), dtype=TYPES[case["dtype"]], device=DEVICE)
    for i in range(e):
        s["b"][i] = _normal(gen, s["b"].shape[1:], k ** -0.5, case["dtype"])
    if case["layout"] == "col":
        s["b"] = s["b"].transpose(1, 2)
    s["bias"] = _normal(gen, (e, n), 0.5, "f32") if case["bias"] else None
    s["grad"] = _normal(gen, (m, n), 1.0, case["dtype"]) if case["step"] else None
    return s


# --- the plain forms -----------------------------------------------------------

def _blocks(x):
    """x (r, k) in 32 bits as blocks (r, kp / 32, 32), zeros past k."""
    r, k = x.shape
    kp = -(-k // 128) * 128
    full = torch.zeros((r, kp), dtype=torch.float32, device=x.device)
    full[:, :k] = x
    return full.view(r, kp // 32, 32)


def _power(exponent):
    """2^exponent in 32 bits, from two factors whose bits are set: exact, from 2^-149 to 2^127."""
    half = exponent >> 1
    return ((half + 127) << 23).view(torch.float32) * ((exponent - half + 127) << 23).view(torch.float32)


def _magnitudes(x):
    """Blocks of x, the exponent of each block's scale, and each value's index in E2M1 (ties to the even code)."""
    blocks = _blocks(x)
    field = blocks.abs().amax(-1).view(torch.int32) >> 23          # the largest magnitude's exponent, biased by 127
    exponent = (field - 127 - 2).clamp(min=-127)                   # 6 = 1.5 * 2^2 is the largest code
    a = blocks.abs() * _power(-exponent).unsqueeze(-1)
    index = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
             + (a >= 3.5).int() + (a > 5.0).int())
    return blocks, exponent, index


def _rounded(x):
    """What x's 4-bit form stands for, in 32 bits."""
    blocks, exponent, index = _magnitudes(x)
    table = torch.tensor(E2M1, device=x.device)
    values = table[index] * _power(exponent).unsqueeze(-1)
    return torch.where(blocks < 0, -values, values).reshape(x.shape[0], -1)[:, : x.shape[1]]


def _encode(x):
    """Codes and scales of x (r, k)."""
    blocks, exponent, index = _magnitudes(x)
    code = (index + 8 * (blocks < 0).int()).to(torch.uint8).reshape(x.shape[0], -1)
    codes = code[:, 0::2] | (code[:, 1::2] << 4)
    scales = (exponent + 127).to(torch.uint8)
    return codes.contiguous(), scales.view(x.shape[0], -1, 4).transpose(0, 1).contiguous()


def _decode(codes, scales, k):
    """The values that codes (..., r, kp / 2) and scales (..., kp / 128, r, 4) stand for, in 32 bits."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    pairs = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()
    per_row = scales.transpose(-3, -2).flatten(-2).int()
    values = table[pairs].unflatten(-1, (-1, 32)) * _power(per_row - 127).unsqueeze(-1)
    return values.flatten(-2)[..., :k]


def _slots(offsets, m):
    """The expert of each row, and the row's place among the expert's rows."""
    row = torch.arange(m, device=offsets.device)
    expert = (row.unsqueeze(1) >= offsets[1:].unsqueeze(0)).sum(1)
    return expert, row - offsets[expert]


def _padded(x, expert, place, groups, longest):
    full = torch.zeros((groups, longest, x.shape[1]), dtype=torch.float32, device=x.device)
    full[expert, place] = x.float()
    return full


def _gelu(x):
    return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))


def _plain_grouped(s):
    case = s["case"]
    expert, place = _slots(s["offsets"], case["m"])
    a = _padded(s["a"], expert, place, case["groups"], s["longest"])
    b = s["b"].float()
    c = torch.bmm(a, b)[expert, place]
    if s["bias"] is not None:
        c = c + s["bias"][expert]
    if case["act"] != "none":
        c = c.clamp(min=0.0) if case["act"] == "relu" else _gelu(c)
    out = {"c": c.to(s["a"].dtype)}
    if case["step"]:
        grad = _padded(s["grad"], expert, place, case["groups"], s["longest"])
        out["da"] = torch.bmm(grad, b.transpose(1, 2))[expert, place].to(s["a"].dtype)
        out["db"] = torch.bmm(a.transpose(1, 2), grad).to(s["a"].dtype)
    return out


def _plain_mx4(s):
    case = s["case"]
    x, w = _rounded(s["a"].float()), _decode(s["codes"], s["scales"], case["k"])
    if not case["groups"]:
        return (x @ w.t()).to(s["a"].dtype)
    expert, place = _slots(s["offsets"], case["m"])
    y = torch.bmm(_padded(x, expert, place, case["groups"], s["longest"]), w.transpose(1, 2))
    return y[expert, place].to(s["a"].dtype)


def _plain_pack(s):
    x = s["x"].float()
    if s["case"]["along"] == "columns":
        x = x.t()
    return _rounded(x).to(s["x"].dtype)


def _plain_route(s):
    case = s["case"]
    e, c = case["groups"], case["choices"]
    x = s["logits"].float()
    ordered, which = torch.sort(x, dim=1, descending=True, stable=True)
    top, which = ordered[:, :c], which[:, :c]
    used = top > float("-inf")
    largest = torch.where(used[:, :1], top[:, :1], torch.zeros_like(top[:, :1]))
    p = torch.exp(x - largest)
    chosen = torch.exp(top - largest)
    total = (chosen if case["normalize"] else p).sum(1, keepdim=True)
    safe = torch.where(total > 0, total, torch.ones_like(total))
    weights = chosen / safe
    experts = torch.where(used, which, torch.full_like(which, -1))
    flat = torch.where(used, which, torch.full_like(which, e)).reshape(-1)
    order = torch.sort(flat, stable=True)[1]
    counts = (flat.unsqueeze(1) == torch.arange(e, device=x.device)).sum(0)
    offsets = torch.cat((counts.new_zeros(1), counts.cumsum(0)))
    place = torch.arange(flat.numel(), device=x.device)
    order = torch.where(place < offsets[-1], order, torch.full_like(order, -1))
    out = {"weights": weights, "experts": experts.int(), "offsets": offsets.int(), "order": order.int()}
    if case["step"]:
        # d weights / d logits of a softmax: w (g - sum w g) over the experts that it sums over.
        grad = torch.where(used, s["grad"], torch.zeros_like(s["grad"]))
        spread = torch.zeros_like(x).scatter_add_(1, which, grad)
        dot = (weights * grad).sum(1, keepdim=True)
        if case["normalize"]:
            share = torch.zeros_like(x).scatter_add_(1, which, torch.where(used, weights, torch.zeros_like(weights)))
        else:
            share = p / safe
        out["dlogits"] = (share * (spread - dot)).to(s["logits"].dtype)
    return out


PLAIN = {"grouped": _plain_grouped, "mx4": _plain_mx4, "pack": _plain_pack, "route": _plain_route}


# --- the library's calls -------------------------------------------------------

def _own_grouped(s):
    import dense_gemm_optimisation_fp32_amd as g

    case = s["case"]
    out = {"c": g.grouped_linear(s["a"], s["b"], s["offsets"], bias=s["bias"], activation=case["act"])}
    if case["step"]:
        out["da"] = g.grouped_linear(s["grad"], s["b"].transpose(1, 2), s["offsets"])
        out["db"] = g.grouped_weight_grad(s["a"], s["grad"], s["offsets"])
    return out


def _own_mx4(s):
    import dense_gemm_optimisation_fp32_amd as g

    w = g.Mx4Tensor(s["codes"], s["scales"], s["case"]["k"])
    return g.mx4_linear(s["a"], w, offsets=s["offsets"])


def _own_pack(s):
    import dense_gemm_optimisation_fp32_amd as g

    x = s["x"] if s["case"]["along"] == "rows" else s["x"].t()
    return g.mx4_dequantize(g.mx4_quantize(x), dtype=x.dtype)


def _own_route(s):
    import dense_gemm_optimisation_fp32_amd as g

    case = s["case"]
    r = g.route(s["logits"], case["choices"], normalize=case["normalize"])
    out = {"weights": r.weights, "experts": r.experts, "offsets": r.offsets, "order": r.order}
    if case["step"]:
        out["dlogits"] = g.route_grad(s["logits"], r, s["grad"])
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"grouped": _own_grouped, "mx4": _own_mx4, "pack": _own_pack, "route": _own_route}[op](state)
    return PLAIN[op](state)


# --- what each pass cannot do without --------------------------------------------

def _experts_used(case):
    """How many experts get a row, on average."""
    e = case["groups"]
    return e * (1.0 - (1.0 - 1.0 / e) ** case["m"])


def work(case):
    size = 2 if case.get("dtype") == "bf16" else 4
    if case["op"] == "route":
        t, e, c = case["tokens"], case["groups"], case["choices"]
        passes = 3 if case["step"] else 1                       # the gradient reads the logits and writes its own
        return {"bytes": passes * t * e * size + (16 if case["step"] else 12) * t * c + 4 * (e + 1),
                "flops": 4 * t * e * (2 if case["step"] else 1)}
    if case["op"] == "pack":
        return {"bytes": 2 * case["rows"] * case["k"] * size, "flops": 4 * case["rows"] * case["k"]}
    m, n, k = case["m"], case["n"], case["k"]
    if case["op"] == "mx4":
        experts = _experts_used(case) if case["groups"] else 1
        return {"bytes": m * (k + n) * size + experts * n * k * 17 / 32, "flops": 2 * m * n * k}
    rows = m * (k + n) * (2 if case["step"] else 1)
    weights = _experts_used(case) * n * k + (case["groups"] * n * k if case["step"] else 0)
    return {"bytes": (rows + weights) * size, "flops": 2 * m * n * k * (3 if case["step"] else 1)}


# --- the definitions in 64 bits ----------------------------------------------------

def _exact_power(exponent):
    return ((exponent.long() + 1023) << 52).view(torch.float64)


def _exact_values(x):
    """x (r, k) rounded to 4 bits with a power of two for each 32 columns, by search over the grid."""
    r, k = x.shape
    out = torch.zeros_like(x, dtype=torch.float64)
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    order = (0, 2, 4, 6, 1, 3, 5, 7)     # of two codes as near, the even one
    for start in range(0, k, 32):
        block = x[:, start:start + 32].double()
        top = block.abs().amax(1, keepdim=True)
        _, exponent = torch.frexp(top)   # top = f * 2^exponent, f in [1/2, 1)
        scale = _exact_power(torch.where(top > 0, (exponent - 3).clamp(min=-127), torch.zeros_like(exponent)))
        a = block.abs() / scale
        best = torch.zeros_like(a)
        far = torch.full_like(a, math.inf)
        for i in order:
            d = (a - grid[i]).abs()
            best = torch.where(d < far, grid[i], best)
            far = torch.minimum(d, far)
        out[:, start:start + 32] = torch.sign(block) * best * scale
    return out


def _exact_weights(codes, scales, k):
    """One matrix's values from its codes and scales."""
    r = codes.shape[0]
    out = torch.zeros((r, codes.shape[1] * 2), dtype=torch.float64, device=codes.device)
    for half in range(2):
        c = (codes >> (4 * half)) & 15
        low, two = (c & 1).double(), (c >> 1) & 3
        size = torch.where(two == 0, low / 2, (1 + low / 2) * _exact_power(two.int() - 1))
        out[:, half::2] = torch.where(c >= 8, -size, size)
    power = _exact_power(scales.permute(1, 0, 2).reshape(r, -1).int() - 127)
    return (out * power.repeat_interleave(32, 1))[:, :k]


def _exact_route(s):
    case = s["case"]
    x = s["logits"].double()
    out = {"weights": None, "experts": None, "offsets": None, "order": None}
    left = x.clone()
    picks = []
    for _ in range(case["choices"]):
        best = left.amax(1, keepdim=True)
        index = torch.where(left == best, torch.arange(x.shape[1], device=x.device), x.shape[1]).amin(1, keepdim=True)
        picks.append((index, torch.isfinite(best)))
        left.scatter_(1, index, -math.inf)
    index = torch.cat([p[0] for p in picks], 1)
    used = torch.cat([p[1] for p in picks], 1)
    index = torch.where(used, index, torch.zeros_like(index))
    chosen = torch.zeros(x.shape, dtype=torch.bool, device=x.device)
    for j in range(case["choices"]):
        chosen |= (torch.arange(x.shape[1], device=x.device) == index[:, j:j + 1]) & used[:, j:j + 1]
    over = torch.where(chosen, x, torch.full_like(x, -math.inf)) if case["normalize"] else x
    p = torch.nan_to_num(torch.softmax(over, 1), nan=0.0)
    out["weights"] = torch.where(used, p.gather(1, index), torch.zeros_like(used, dtype=torch.float64))
    if case["step"]:
        g = torch.zeros_like(x)
        g.scatter_add_(1, index, torch.where(used, s["grad"].double(), torch.zeros_like(out["weights"])))
        out["dlogits"] = p * (g - (p * g).sum(1, keepdim=True))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(s)
    if case["op"] == "pack":
        x = s["x"] if case["along"] == "rows" else s["x"].t()
        return _exact_values(x)
    m, n = case["m"], case["n"]
    ends = s["offsets"].tolist() if case["groups"] else [0, m]
    if case["op"] == "mx4":
        x = _exact_values(s["a"])
        y = torch.zeros((m, n), dtype=torch.float64, device=DEVICE)
        for e in range(len(ends) - 1):
            codes, scales = (s["codes"][e], s["scales"][e]) if case["groups"] else (s["codes"], s["scales"])
            rows = slice(ends[e], ends[e + 1])
            y[rows] = torch.mm(x[rows], _exact_weights(codes, scales, case["k"]).t())
        return y
    out = {"c": torch.zeros((m, n), dtype=torch.float64, device=DEVICE)}
    if case["step"]:
        out["da"] = torch.zeros((m, case["k"]), dtype=torch.float64, device=DEVICE)
        out["db"] = torch.zeros((case["groups"], case["k"], n), dtype=torch.float64, device=DEVICE)
    for e in range(len(ends) - 1):
        rows = slice(ends[e], ends[e + 1])
        a, b = s["a"][rows].double(), s["b"][e].double()
        c = torch.mm(a, b)
        if s["bias"] is not None:
            c += s["bias"][e].double()
        if case["act"] == "relu":
            c = torch.relu(c)
        elif case["act"] == "gelu":
            c = c * torch.special.ndtr(c)
        out["c"][rows] = c
        if case["step"]:
            grad = s["grad"][rows].double()
            out["da"][rows] = torch.mm(grad, b.t())
            out["db"][e] = torch.mm(a.t(), grad)
    return out
