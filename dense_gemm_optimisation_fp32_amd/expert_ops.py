"""Python binding of the expert-layer operators (include/expert_ops.h): routing,
products grouped by expert with their gradients, and microscaled 4-bit
quantisation and products.

Argument marshalling only, as in the package's ``matmul`` and ``linear``: every
step runs in the library's HIP kernels on the current stream, results and
workspaces come from PyTorch's allocator, a failed call raises
``GemmF32Error`` and there is no fallback.

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

from . import (_ACTIVATIONS, GEMM_F32_COL_MAJOR, GEMM_F32_ROW_MAJOR, GEMM_F32_SUCCESS, GemmF32Error,
               load_library)

EXPERT_F32 = 0
EXPERT_BF16 = 1
_DTYPES = {torch.float32: EXPERT_F32, torch.bfloat16: EXPERT_BF16}

EXPERT_FUNCTIONS = (
    "expert_grouped_linear", "expert_grouped_weight_grad", "expert_mx4_quantize", "expert_mx4_dequantize",
    "expert_mx4_workspace", "expert_mx4_linear", "expert_route_workspace", "expert_route", "expert_route_grad",
)

_fns = None
_raw_stream = torch._C._cuda_getCurrentRawStream     # current_stream(device).cuda_stream in a tenth of its time
_current_device = torch._C._cuda_getDevice


def _functions():
    """The entry points on integers, {name: function}, bound once."""
    global _fns
    if _fns is None:
        lib = load_library()
        try:
            from . import _expert_binding
        except ImportError as e:
            raise RuntimeError("_expert_binding.so is not built; run __graft_entry__.build() or "
                               "python -m dense_gemm_optimisation_fp32_amd.build") from e
        _expert_binding.bind({name: ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
                              for name in EXPERT_FUNCTIONS})
        _fns = {name: getattr(_expert_binding, name) for name in EXPERT_FUNCTIONS}
    return _fns


def _call(name, index, *args):
    """Entry point `name` on device `index` and its current stream, the last argument."""
    fn = (_fns or _functions())[name]
    if index == _current_device():
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, _raw_stream(index))
    if st != GEMM_F32_SUCCESS:
        raise GemmF32Error(st, name)


def _dtype(x, what):
    d = _DTYPES.get(x.dtype)
    if d is None:
        raise TypeError(f"{what} must be float32 or bfloat16")
    return d


def _on(device, **tensors):
    for what, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{what} must be on {device}")


def _gpu(x, what):
    if not x.is_cuda:
        raise ValueError(f"{what} must be on a GPU")


def _rows(x, what):
    """Distance between the rows of a 2-D tensor with unit stride along its columns."""
    if x.dim() != 2:
        raise ValueError(f"{what} must be 2-D")
    if x.shape[1] > 1 and x.stride(1) != 1:
        raise ValueError(f"{what} needs unit stride along its rows")
    if x.shape[0] > 1:
        ld = x.stride(0)
        if ld < x.shape[1]:
            raise ValueError(f"{what} has overlapping rows")
        return ld
    return x.shape[1]


def _offsets(offsets, groups, device):
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or offsets.numel() != groups + 1 or not offsets.is_contiguous():
        raise ValueError(f"offsets must be {groups + 1} contiguous int32 values")
    _on(device, offsets=offsets)


def _bias(bias, groups, n, device):
    if bias is None:
        return None
    if bias.dtype != torch.float32 or tuple(bias.shape) != (groups, n) or not bias.is_contiguous():
        raise ValueError(f"bias must be a contiguous float32 ({groups}, {n}) tensor")
    _on(device, bias=bias)
    return bias.data_ptr()


def _out(out, shape, dtype, device):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if tuple(out.shape) != shape or out.dtype != dtype or out.device != device:
        raise ValueError(f"out must be a {dtype} {shape} tensor on {device}")
    return out


def grouped_linear(a: torch.Tensor, b: torch.Tensor, offsets: torch.Tensor, bias: torch.Tensor | None = None,
                   activation=None, out: torch.Tensor | None = None) -> torch.Tensor:
    """act(a_e . b_e + bias_e) for every expert e.

    a: (m, k) float32 or bfloat16, rows sorted by expert; b: (groups, k, n) of
    a's type, unit stride along n or (transposed weights) along k; offsets:
    groups + 1 int32, expert e's rows are offsets[e] .. offsets[e + 1]; bias:
    (groups, n) float32.  Rows of no expert become zero.  The gradient with
    respect to a is ``grouped_linear(grad, b.transpose(1, 2), offsets)``."""
    dt = _dtype(a, "a")
    _gpu(a, "a")
    lda = _rows(a, "a")
    if b.dim() != 3:
        raise ValueError("b must be 3-D")
    if b.dtype != a.dtype:
        raise TypeError("a and b must have the same type")
    m, k = a.shape
    groups, k2, n = b.shape
    if k != k2:
        raise ValueError(f"inner dimensions differ: a is {tuple(a.shape)}, b is {tuple(b.shape)}")
    device = a.device
    se, sk, sn = b.stride()
    if sn == 1 or n == 1:
        layout, ldb, least = GEMM_F32_ROW_MAJOR, (sk if k > 1 else n), n
        if sn != 1 and sk == 1:
            layout, ldb, least = GEMM_F32_COL_MAJOR, max(sn, k), k
    elif sk == 1 or k == 1:
        layout, ldb, least = GEMM_F32_COL_MAJOR, sn, k
    else:
        raise ValueError("b needs unit stride along n or along k")
    if ldb < least:
        raise ValueError("b has overlapping rows")
    _on(device, b=b)
    _offsets(offsets, groups, device)
    bias_ptr = _bias(bias, groups, n, device)
    out = _out(out, (m, n), a.dtype, device)
    ldc = _rows(out, "out")
    _call("expert_grouped_linear", device.index, dt, m, n, k, groups, a.data_ptr(), lda, b.data_ptr(), layout, ldb,
          se, offsets.data_ptr(), bias_ptr, _ACTIVATIONS[activation], out.data_ptr(), ldc)
    return out


def grouped_weight_grad(a: torch.Tensor, grad: torch.Tensor, offsets: torch.Tensor,
                        out: torch.Tensor | None = None) -> torch.Tensor:
    """a_e^T . grad_e for every expert e: (groups, k, n) from a (m, k) and grad
    (m, n), rows sorted by expert; zero for an expert without rows."""
    dt = _dtype(a, "a")
    _gpu(a, "a")
    lda, ldg = _rows(a, "a"), _rows(grad, "grad")
    if grad.dtype != a.dtype:
        raise TypeError("a and grad must have the same type")
    if grad.shape[0] != a.shape[0]:
        raise ValueError(f"row counts differ: a is {tuple(a.shape)}, grad is {tuple(grad.shape)}")
    device = a.device
    _on(device, grad=grad)
    groups = offsets.numel() - 1
    _offsets(offsets, groups, device)
    m, k = a.shape
    n = grad.shape[1]
    out = _out(out, (groups, k, n), a.dtype, device)
    se, ldd, sn = out.stride()
    if (n > 1 and sn != 1) or (k > 1 and ldd < n):
        raise ValueError("out needs unit stride along its rows")
    if k == 1:
        ldd = n
    _call("expert_grouped_weight_grad", device.index, dt, m, n, k, groups, a.data_ptr(), lda, grad.data_ptr(), ldg,
          offsets.data_ptr(), out.data_ptr(), ldd, se)
    return out


def _blocks(k):
    return (k + 127) // 128


class Mx4Tensor:
    """Matrices in microscaled 4-bit floating point: ``codes`` (..., r, kp / 2)
    and ``scales`` (..., kp / 128, r, 4), uint8, for r rows of k columns (kp = k
    rounded up to 128); a leading dimension holds one matrix an expert."""

    __slots__ = ("codes", "scales", "k")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, k: int):
        kb = _blocks(k)
        if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise TypeError("codes and scales must be uint8")
        if k < 1 or codes.dim() not in (2, 3) or scales.dim() != codes.dim() + 1:
            raise ValueError("codes must be (r, kp / 2) or (groups, r, kp / 2), scales (kp / 128, r, 4) in each")
        if codes.shape[-1] != kb * 64 or tuple(scales.shape) != (*codes.shape[:-2], kb, codes.shape[-2], 4):
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
    dt = _dtype(x, "x")
    _gpu(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    r, k = x.shape
    if k < 1:
        raise ValueError("x needs at least one column")
    if x.stride(1) == 1 or k == 1 or r == 0:
        layout, ld = GEMM_F32_ROW_MAJOR, (x.stride(0) if r > 1 else k)
        if r > 1 and k == 1 and x.stride(0) == 1:
            ld = 1
        least = k
    elif x.stride(0) == 1 or r == 1:
        layout, ld, least = GEMM_F32_COL_MAJOR, x.stride(1), r
    else:
        raise ValueError("x needs unit stride along one axis")
    if ld < least:
        raise ValueError("x has overlapping rows")
    kb = _blocks(k)
    codes = torch.empty((r, kb * 64), dtype=torch.uint8, device=x.device)
    scales = torch.empty((kb, r, 4), dtype=torch.uint8, device=x.device)
    _call("expert_mx4_quantize", x.device.index, dt, r, k, x.data_ptr(), layout, ld, codes.data_ptr(),
          scales.data_ptr())
    q = Mx4Tensor.__new__(Mx4Tensor)          # (checked by construction)
    q.codes, q.scales, q.k = codes, scales, k
    return q


def mx4_dequantize(q: Mx4Tensor, dtype: torch.dtype = torch.float32, out: torch.Tensor | None = None) -> torch.Tensor:
    """The values that one matrix's codes stand for, (r, k) of ``dtype`` (exact in both types)."""
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise TypeError("dtype must be float32 or bfloat16")
    if q.codes.dim() != 2:
        raise ValueError("q must hold one matrix")
    _gpu(q.codes, "q")
    r = q.codes.shape[0]
    out = _out(out, (r, q.k), dtype, q.device)
    ld = _rows(out, "out")
    _call("expert_mx4_dequantize", q.device.index, dt, r, q.k, q.codes.data_ptr(), q.scales.data_ptr(),
          out.data_ptr(), ld)
    return out


def mx4_linear(x: torch.Tensor, w: Mx4Tensor, offsets: torch.Tensor | None = None, bias: torch.Tensor | None = None,
               activation=None, out: torch.Tensor | None = None) -> torch.Tensor:
    """act(Q(x) . W^T + bias): x (m, k) is quantised to 4 bits on the way, w holds
    W (n, k), or with offsets (groups + 1 int32) one W an expert for x's rows
    sorted by expert.  bias: (n) or (groups, n) float32.  The result has x's type."""
    dt = _dtype(x, "x")
    _gpu(x, "x")
    ldx = _rows(x, "x")
    m, k = x.shape
    if k != w.k:
        raise ValueError(f"inner dimensions differ: x is {tuple(x.shape)}, w is {tuple(w.shape)}")
    device = x.device
    _on(device, w=w.codes)
    n = w.codes.shape[-2]
    if w.codes.dim() == 3:
        groups = w.codes.shape[0]
        if offsets is None:
            raise ValueError("one matrix an expert needs offsets")
        _offsets(offsets, groups, device)
        offsets_ptr = offsets.data_ptr()
    else:
        groups, offsets_ptr = 1, None
        if offsets is not None:
            raise ValueError("offsets need one matrix an expert")
        if bias is not None and bias.dim() == 1:
            bias = bias.unsqueeze(0)
    bias_ptr = _bias(bias, groups, n, device)
    out = _out(out, (m, n), x.dtype, device)
    ldy = _rows(out, "out")
    need = _functions()["expert_mx4_workspace"](m, n, k, groups)
    space = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    _call("expert_mx4_linear", device.index, dt, m, n, k, groups, x.data_ptr(), ldx, w.codes.data_ptr(),
          w.scales.data_ptr(), offsets_ptr, bias_ptr, _ACTIVATIONS[activation], out.data_ptr(), ldy,
          space.data_ptr() if need else None, need)
    return out


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
    dt = _dtype(logits, "logits")
    _gpu(logits, "logits")
    ld = _rows(logits, "logits")
    tokens, groups = logits.shape
    if not 1 <= choices <= groups:
        raise ValueError(f"choices must be from 1 to the {groups} experts")
    device = logits.device
    weights = torch.empty((tokens, choices), dtype=torch.float32, device=device)
    experts = torch.empty((tokens, choices), dtype=torch.int32, device=device)
    offsets = torch.empty(groups + 1, dtype=torch.int32, device=device)
    order = torch.empty(tokens * choices, dtype=torch.int32, device=device)
    need = _functions()["expert_route_workspace"](tokens, groups)
    space = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    _call("expert_route", device.index, dt, tokens, groups, choices, 1 if normalize else 0, logits.data_ptr(), ld,
          weights.data_ptr(), experts.data_ptr(), offsets.data_ptr(), order.data_ptr(),
          space.data_ptr() if need else None, need)
    return Routing(weights, experts, offsets, order, bool(normalize))


def route_grad(logits: torch.Tensor, r: Routing, grad: torch.Tensor) -> torch.Tensor:
    """The logits' gradient from that of r.weights (tokens, choices, float32)."""
    dt = _dtype(logits, "logits")
    _gpu(logits, "logits")
    ld = _rows(logits, "logits")
    tokens, groups = logits.shape
    if r.weights.dim() != 2 or r.weights.shape[0] != tokens or r.experts.shape != r.weights.shape:
        raise ValueError("r is not the routing of these logits")
    if r.weights.dtype != torch.float32 or r.experts.dtype != torch.int32 or not (
            r.weights.is_contiguous() and r.experts.is_contiguous()):
        raise ValueError("r must hold contiguous float32 weights and int32 experts")
    if grad.dtype != torch.float32 or grad.shape != r.weights.shape or not grad.is_contiguous():
        raise ValueError(f"grad must be a contiguous float32 {tuple(r.weights.shape)} tensor")
    device = logits.device
    _on(device, weights=r.weights, experts=r.experts, grad=grad)
    out = torch.empty((tokens, groups), dtype=logits.dtype, device=device)
    _call("expert_route_grad", device.index, dt, tokens, groups, r.weights.shape[1], 1 if r.normalize else 0,
          logits.data_ptr(), ld, r.weights.data_ptr(), r.experts.data_ptr(), grad.data_ptr(), out.data_ptr(), groups)
    return out
