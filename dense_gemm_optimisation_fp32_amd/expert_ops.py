"""Python binding of the expert-layer operators (include/expert_ops.h): routing,
products grouped by expert with their gradients, and microscaled 4-bit
quantisation and products.

Argument marshalling only, as in the package's ``matmul`` and ``linear`` (in C++,
csrc/expert_binding.cpp, because the calls are short): every step runs in the
library's HIP kernels on the current stream, results and workspaces come from
PyTorch's allocator, and there is no fallback.  Wrong arguments raise
``TypeError`` or ``ValueError``, an activation that there is not ``KeyError``;
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
"""
from __future__ import annotations

import ctypes

import torch

from . import _ACTIVATIONS, GemmF32Error, load_library

EXPERT_F32 = 0
EXPERT_BF16 = 1
_DTYPES = {torch.float32: EXPERT_F32, torch.bfloat16: EXPERT_BF16}

EXPERT_FUNCTIONS = (
    "expert_grouped_linear", "expert_grouped_weight_grad", "expert_mx4_quantize", "expert_mx4_dequantize",
    "expert_mx4_workspace", "expert_mx4_linear", "expert_route_workspace", "expert_route", "expert_route_grad",
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
        i64, i32, vp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
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
    if x.dtype not in _DTYPES and x.dtype != torch.uint8:
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
