"""Python binding of the expert-layer operators (include/expert_ops.h): routing,
products grouped by expert with their gradients, microscaled 4-bit and 8-bit
integer quantisation and products, and orthogonalised updates.

Argument marshalling only, as in the package's ``matmul`` and ``linear`` (in C++,
csrc/expert_binding.cpp, because the calls are short): every step runs in the
library's HIP kernels on the current stream, results and workspaces come from
PyTorch's allocator, and there is no fallback.  Wrong arguments raise
``TypeError`` or ``ValueError``, an activation or scores that there are not ``KeyError``;
``GemmF32Error`` is what the library itself refuses (sizes outside the limits of
expert_ops.h, more than 32 choices among them) or fails at.  Results carry no
autograd history, whatever the operands' ``requires_grad``: the gradients are
the calls below.

    r = g.route(logits, choices=2)                      # tokens -> experts
    a = x[r.order.clamp(min=0) // 2]                    # rows sorted by expert
    h = g.grouped_linear(a, w1, r.offsets, bias=b1, activation="gelu")
    dw = g.grouped_weight_grad(a, dh, r.offsets)        # gradients
    q = g.mx4_quantize(w)                               # w (n, k) in 4 bits
    y = g.mx4_linear(x, q)                              # Q(x) . W^T
    r = g.route_balanced(logits, 8, bias=b, sets=8, kept_sets=4)
    q = g.int8_quantize(w)                              # w (n, k) in 8 bits, a scale a row
    y = g.int8_linear(x, q, bias=b1, activation="gelu")
    w1 -= rate * g.orthogonalize(dw)                    # an update an expert
"""
from __future__ import annotations

import ctypes
import numbers
import operator

import torch

from . import _ACTIVATIONS, GemmF32Error, load_library

EXPERT_F32 = 0
EXPERT_BF16 = 1
EXPERT_SIGMOID = 0
EXPERT_SOFTMAX = 1
_SCORES = {"sigmoid": EXPERT_SIGMOID, "softmax": EXPERT_SOFTMAX}
_DTYPES = {torch.float32: EXPERT_F32, torch.bfloat16: EXPERT_BF16}

EXPERT_FUNCTIONS = (
    "expert_grouped_linear", "expert_grouped_weight_grad", "expert_mx4_quantize", "expert_mx4_dequantize",
    "expert_mx4_workspace", "expert_mx4_linear", "expert_route_workspace", "expert_route", "expert_route_grad",
    "expert_route_balanced_workspace", "expert_route_balanced", "expert_route_balanced_grad", "expert_int8_quantize",
    "expert_int8_dequantize", "expert_int8_workspace", "expert_int8_linear", "expert_orthogonalize_workspace",
    "expert_orthogonalize",
)

_fns = None
_module = None
# current_stream(device).cuda_stream in a tenth of its time (None: a torch
# without GPU support, which has no tensors to ask for).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _functions():
    """The C entry points with their signatures, set once."""
    global _fns
    if _fns is None:
        lib = load_library()
        i64, i32, vp, f32 = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_float
        signatures = {
            "expert_grouped_linear": ([i32, i64, i64, i64, i64, vp, i64, vp, i32, i64, i64, vp, vp, i32, vp, i64, vp], i32),
            "expert_grouped_weight_grad": ([i32, i64, i64, i64, i64, vp, i64, vp, i64, vp, vp, i64, i64, vp], i32),
            "expert_mx4_quantize": ([i32, i64, i64, vp, i32, i64, vp, vp, vp], i32),
            "expert_mx4_dequantize": ([i32, i64, i64, vp, vp, vp, i64, vp], i32),
            "expert_mx4_workspace": ([i64, i64, i64, i64], i64),
            "expert_mx4_linear": ([i32, i64, i64, i64, i64, vp, i64, vp, vp, vp, vp, i32, vp, i64, vp, i64, vp], i32),
            "expert_route_workspace": ([i64, i64], i64),
            "expert_route": ([i32, i64, i64, i64, i32, vp, i64, vp, vp, vp, vp, vp, i64, vp], i32),
            "expert_route_grad": ([i32, i64, i64, i64, i32, vp, i64, vp, vp, vp, vp, i64, vp], i32),
            "expert_route_balanced_workspace": ([i64, i64], i64),
            "expert_route_balanced": ([i32, i64, i64, i64, i32, i64, i64, i32, f32, vp, i64, vp, vp, vp, vp, vp, vp, i64, vp], i32),
            "expert_route_balanced_grad": ([i32, i64, i64, i64, i32, i32, f32, vp, i64, vp, vp, vp, vp, i64, vp], i32),
            "expert_int8_quantize": ([i32, i64, i64, vp, i32, i64, vp, vp, vp], i32),
            "expert_int8_dequantize": ([i32, i64, i64, vp, vp, vp, i64, vp], i32),
            "expert_int8_workspace": ([i64, i64], i64),
            "expert_int8_linear": ([i32, i64, i64, i64, i64, vp, i64, vp, vp, vp, vp, i32, vp, i64, vp, i64, vp], i32),
            "expert_orthogonalize_workspace": ([i32, i64, i64, i64], i64),
            "expert_orthogonalize": ([i32, i64, i64, i64, vp, i64, i64, i32, vp, f32, vp, i64, i64, vp, i64, vp], i32),
        }
        fns = {}
        for name, (args, res) in signatures.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
            fns[name] = fn
        _fns = fns
    return _fns


def _binding():
    """The compiled module in front of them, bound once."""
    global _module
    if _module is None:
        addresses = {name: ctypes.cast(fn, ctypes.c_void_p).value for name, fn in _functions().items()}
        try:
            from . import _expert_binding
        except ImportError as e:
            raise RuntimeError("_expert_binding is not built for this Python or does not load; run __graft_entry__.build() or "
                               "python -m dense_gemm_optimisation_fp32_amd.build") from e
        _expert_binding.bind(addresses)
        _module = _expert_binding
    return _module


def _stream(x, what):
    """The current stream of x's device."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{what} must be a tensor")
    if x.is_cuda:
        return _raw_stream(x.device.index)
    if x.dtype not in _DTYPES and x.dtype not in (torch.uint8, torch.int8):
        raise TypeError(f"{what} must be float32 or bfloat16")
    raise ValueError(f"{what} must be on a GPU")


def _checked(result, name):
    if type(result) is int:
        raise GemmF32Error(result, name)
    return result


def grouped_linear(a: torch.Tensor, b: torch.Tensor, offsets: torch.Tensor, bias: torch.Tensor | None = None,
                   activation=None, out: torch.Tensor | None = None) -> torch.Tensor:
    """act(a_e . b_e + bias_e) for every expert e.

    a: (m, k) float32 or bfloat16, rows sorted by expert; b: (groups, k, n) of
    a's type, unit stride along n or (transposed weights) along k; offsets:
    groups + 1 int32, expert e's rows are offsets[e] .. offsets[e + 1]; bias:
    (groups, n) float32.  Rows of no expert become zero.  The gradient with
    respect to a is ``grouped_linear(grad, b.transpose(1, 2), offsets)``."""
    return _checked((_module or _binding()).grouped_linear(a, b, offsets, bias, _ACTIVATIONS[activation], out,
                                                           _stream(a, "a")), "expert_grouped_linear")


def grouped_weight_grad(a: torch.Tensor, grad: torch.Tensor, offsets: torch.Tensor,
                        out: torch.Tensor | None = None) -> torch.Tensor:
    """a_e^T . grad_e for every expert e: (groups, k, n) from a (m, k) and grad
    (m, n), rows sorted by expert; zero for an expert without rows."""
    return _checked((_module or _binding()).grouped_weight_grad(a, grad, offsets, out, _stream(a, "a")),
                    "expert_grouped_weight_grad")


class Mx4Tensor:
    """Matrices in microscaled 4-bit floating point: ``codes`` (..., r, kp / 2)
    and ``scales`` (..., kp / 128, r, 4), uint8, for r rows of k columns (kp = k
    rounded up to 128); a leading dimension holds one matrix an expert."""

    __slots__ = ("codes", "scales", "k")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, k: int):
        kb = (k + 127) // 128
        if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise TypeError("codes and scales must be uint8")
        shape = codes.shape
        if k < 1 or len(shape) not in (2, 3) or scales.dim() != len(shape) + 1:
            raise ValueError("codes must be (r, kp / 2) or (groups, r, kp / 2), scales (kp / 128, r, 4) in each")
        if shape[-1] != kb * 64 or scales.shape != (*shape[:-2], kb, shape[-2], 4):
            raise ValueError(f"codes {tuple(codes.shape)} and scales {tuple(scales.shape)} do not hold {k} columns")
        if not (codes.is_contiguous() and scales.is_contiguous()) or codes.device != scales.device:
            raise ValueError("codes and scales must be contiguous and on one device")
        self.codes, self.scales, self.k = codes, scales, k

    @property
    def shape(self):
        return torch.Size((*self.codes.shape[:-1], self.k))

    @property
    def device(self):
        return self.codes.device


def mx4_quantize(x: torch.Tensor) -> Mx4Tensor:
    """x (r, k), float32 or bfloat16 with unit stride along either axis, in 4
    bits: blocks of 32 along k share a power of two."""
    codes, scales = _checked((_module or _binding()).mx4_quantize(x, _stream(x, "x")), "expert_mx4_quantize")
    q = Mx4Tensor.__new__(Mx4Tensor)          # (they fit by construction)
    q.codes, q.scales, q.k = codes, scales, x.shape[1]
    return q


def mx4_dequantize(q: Mx4Tensor, dtype: torch.dtype = torch.float32, out: torch.Tensor | None = None) -> torch.Tensor:
    """The values that one matrix's codes stand for, (r, k) of ``dtype`` (exact in both types)."""
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise TypeError("dtype must be float32 or bfloat16")
    return _checked((_module or _binding()).mx4_dequantize(q.codes, q.scales, q.k, dt, out, _stream(q.codes, "q")),
                    "expert_mx4_dequantize")


def mx4_linear(x: torch.Tensor, w: Mx4Tensor, offsets: torch.Tensor | None = None, bias: torch.Tensor | None = None,
               activation=None, out: torch.Tensor | None = None) -> torch.Tensor:
    """act(Q(x) . W^T + bias): x (m, k) is quantised to 4 bits on the way, w holds
    W (n, k), or with offsets (groups + 1 int32) one W an expert for x's rows
    sorted by expert.  bias: (n) or (groups, n) float32.  The result has x's type."""
    return _checked((_module or _binding()).mx4_linear(x, w.codes, w.scales, w.k, offsets, bias,
                                                       _ACTIVATIONS[activation], out, _stream(x, "x")),
                    "expert_mx4_linear")


class Routing:
    """What ``route`` returns: ``weights`` and ``experts`` (tokens, choices),
    ``offsets`` (groups + 1), ``order`` (tokens * choices), ``normalize``."""

    __slots__ = ("weights", "experts", "offsets", "order", "normalize")

    def __init__(self, weights, experts, offsets, order, normalize):
        self.weights, self.experts, self.offsets, self.order, self.normalize = weights, experts, offsets, order, normalize


def route(logits: torch.Tensor, choices: int, normalize: bool = True) -> Routing:
    """The `choices` largest logits (tokens, groups) of each token: their softmax
    weights (over the chosen ones, or with normalize false over all), their
    experts (-1 and weight 0 where a token has too few experts that are not at
    -inf), and the slots token * choices + j sorted by expert (``order``, with
    -1 after the last one; expert e's are offsets[e] .. offsets[e + 1])."""
    normalize = bool(normalize)
    found = _checked((_module or _binding()).route(logits, choices, normalize, _stream(logits, "logits")),
                     "expert_route")
    return Routing(*found, normalize)


def route_grad(logits: torch.Tensor, r: Routing, grad: torch.Tensor) -> torch.Tensor:
    """The logits' gradient from that of r.weights (tokens, choices, float32)."""
    return _checked((_module or _binding()).route_grad(logits, r.weights, r.experts, r.normalize, grad,
                                                       _stream(logits, "logits")), "expert_route_grad")


class BalancedRouting(Routing):
    """What ``route_balanced`` returns: as ``Routing``, and ``scores`` and ``scale``."""

    __slots__ = ("scores", "scale")

    def __init__(self, weights, experts, offsets, order, normalize, scores, scale):
        super().__init__(weights, experts, offsets, order, normalize)
        self.scores, self.scale = scores, scale


def route_balanced(logits: torch.Tensor, choices: int, bias: torch.Tensor | None = None, scores: str = "sigmoid", sets: int = 1,
                   kept_sets: int = 1, normalize: bool = True, scale: float = 1.0) -> BalancedRouting:
    """Routing by scores s, "sigmoid" of the logits (tokens, groups) or "softmax"
    over them.  Chosen are the `choices` largest s + bias (groups float32; it
    balances the experts' loads and has no part in the weights), with sets > 1 only
    from the token's `kept_sets` sets of neighbouring experts whose two largest sum
    to the most.  The weights are scale * s / sum of the chosen s, or with
    normalize false scale * s.  Otherwise as ``route``."""
    normalize = bool(normalize)
    found = _checked((_module or _binding()).route_balanced(logits, choices, bias, _SCORES[scores], sets, kept_sets, normalize,
                                                            scale, _stream(logits, "logits")), "expert_route_balanced")
    return BalancedRouting(*found, normalize, scores, scale)


def route_balanced_grad(logits: torch.Tensor, r: BalancedRouting, grad: torch.Tensor) -> torch.Tensor:
    """The logits' gradient from that of r.weights (tokens, choices, float32).
    What is chosen, and so the bias, has no gradient."""
    return _checked((_module or _binding()).route_balanced_grad(logits, r.weights, r.experts, _SCORES[r.scores], r.normalize,
                                                                r.scale, grad, _stream(logits, "logits")),
                    "expert_route_balanced_grad")


class Int8Tensor:
    """Matrices in 8-bit integers with a scale for each row: ``codes`` (..., r,
    kp) int8 and ``scales`` (..., r) float32, for r rows of k columns (kp = k
    rounded up to 16, zeros past k); a leading dimension holds one matrix an
    expert."""

    __slots__ = ("codes", "scales", "k")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, k: int):
        if codes.dtype != torch.int8 or scales.dtype != torch.float32:
            raise TypeError("codes must be int8 and scales float32")
        shape = codes.shape
        if k < 1 or len(shape) not in (2, 3) or scales.shape != shape[:-1]:
            raise ValueError("codes must be (r, kp) or (groups, r, kp), scales (r) or (groups, r)")
        if shape[-1] != (k + 15) // 16 * 16:
            raise ValueError(f"codes {tuple(shape)} do not hold {k} columns")
        if not (codes.is_contiguous() and scales.is_contiguous()) or codes.device != scales.device:
            raise ValueError("codes and scales must be contiguous and on one device")
        self.codes, self.scales, self.k = codes, scales, k

    @property
    def shape(self):
        return torch.Size((*self.codes.shape[:-1], self.k))

    @property
    def device(self):
        return self.codes.device


def int8_quantize(x: torch.Tensor) -> Int8Tensor:
    """x (r, k), float32 or bfloat16 with unit stride along either axis, in 8-bit
    integers: a row's largest magnitude becomes 127."""
    codes, scales = _checked((_module or _binding()).int8_quantize(x, _stream(x, "x")), "expert_int8_quantize")
    q = Int8Tensor.__new__(Int8Tensor)        # (they fit by construction)
    q.codes, q.scales, q.k = codes, scales, x.shape[1]
    return q


def int8_dequantize(q: Int8Tensor, dtype: torch.dtype = torch.float32, out: torch.Tensor | None = None) -> torch.Tensor:
    """The values that one matrix's codes stand for, (r, k) of ``dtype``, rounded once."""
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise TypeError("dtype must be float32 or bfloat16")
    return _checked((_module or _binding()).int8_dequantize(q.codes, q.scales, q.k, dt, out, _stream(q.codes, "q")),
                    "expert_int8_dequantize")


def int8_linear(x: torch.Tensor, w: Int8Tensor, offsets: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                activation=None, out: torch.Tensor | None = None) -> torch.Tensor:
    """act(Q(x) . W^T + bias): x (m, k) is quantised to 8 bits on the way, a scale
    for each row (token), w holds W (n, k), a scale for each row (channel), or with
    offsets (groups + 1 int32) one W an expert for x's rows sorted by expert.  bias:
    (n) or (groups, n) float32.  The result has x's type."""
    return _checked((_module or _binding()).int8_linear(x, w.codes, w.scales, w.k, offsets, bias, _ACTIVATIONS[activation], out,
                                                        _stream(x, "x")), "expert_int8_linear")


def _number(v):
    if isinstance(v, numbers.Real) or (getattr(v, "ndim", None) == 0):
        return float(v)
    raise TypeError


def _coefficients(coefficients, steps):
    """(a, b, c) of every step, one after the other, from one triple or one a step."""
    steps = operator.index(steps)
    if not 1 <= steps <= 64:
        raise ValueError("steps must be from 1 to 64")
    try:
        given = list(coefficients)
        one = not given or isinstance(given[0], numbers.Real) or getattr(given[0], "ndim", None) == 0
        flat = tuple(_number(v) for v in given) if one else tuple(_number(v) for step in given for v in step)
    except TypeError:
        raise TypeError("coefficients must be three numbers, or three for each step") from None
    if one and len(flat) == 3:
        return flat * steps
    if len(flat) != 3 * steps:
        raise ValueError(f"coefficients must be three numbers, or three for each of the {steps} steps")
    return flat


def orthogonalize(x: torch.Tensor, steps: int = 5, coefficients=(3.4445, -4.7750, 2.0315), scale: float = 1.0,
                  out: torch.Tensor | None = None) -> torch.Tensor:
    """scale * x with its singular values brought near one and its singular vectors
    kept, for a matrix (rows, cols) or each of a stack (batch, rows, cols), float32
    or bfloat16 with unit stride along either axis of the matrices.

    From x / |x|, ``steps`` times X <- (a I + b A + c A A) X with A = X X^T, which
    takes a singular value s to a s + b s^3 + c s^5.  Between the products X, A and
    a I + b A + c A A are held in 22 bits, whatever x's type, sums in 32, and the result
    is rounded once.  That is as precise as products of 32-bit matrices, but where singular
    values fall fast (rank 8 over noise of 1e-3: 6.6e-5 off, those 5.2e-5).  ``coefficients``: (a, b, c), or
    one such triple a step.  The result has x's type and unit stride along x's axis, as
    out has to; out may be x."""
    flat = _coefficients(coefficients, steps)
    if isinstance(x, torch.Tensor) and x.dim() in (2, 3) and x.stride(-1) != 1 and x.shape[-1] > 1 and x.stride(-2) == 1:
        if out is not None:
            if not isinstance(out, torch.Tensor):
                raise TypeError("out must be a tensor")
            if out.shape != x.shape:
                raise ValueError(f"out must have x's shape {tuple(x.shape)}")
            if out.shape[-2] > 1 and out.stride(-2) != 1:
                raise ValueError("out needs unit stride along the same axis as x, its columns")
        turned = _orthogonalize(x.transpose(-1, -2), flat, scale, None if out is None else out.transpose(-1, -2))
        return turned.transpose(-1, -2) if out is None else out
    return _orthogonalize(x, flat, scale, out)


def _orthogonalize(x, flat, scale, out):
    return _checked((_module or _binding()).orthogonalize(x, len(flat) // 3, flat, scale, out, _stream(x, "x")), "expert_orthogonalize")
