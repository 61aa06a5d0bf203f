"""What the expert-layer calls report, on the GPU."""
import ctypes

import pytest
import torch

import dense_gemm_optimisation_fp32_amd as g

pytestmark = pytest.mark.gpu

DEV = "cuda"


def hip_runtime():
    """The HIP runtime that this process has loaded."""
    torch.cuda.init()
    with open("/proc/self/maps") as maps:
        return ctypes.CDLL(next(line.split()[-1] for line in maps if "libamdhip64" in line))


def test_an_error_left_by_another_call_is_not_theirs():
    """A HIP call that failed before (a device that there is not) leaves its
    error on the thread; the operators' launches succeed all the same, and it
    is still there for its owner."""
    hip = hip_runtime()
    x = torch.randn((300, 64), device=DEV)
    off = torch.tensor([0, 100, 300], dtype=torch.int32, device=DEV)
    b = torch.randn((2, 64, 96), device=DEV)
    grad = torch.randn((300, 4), device=DEV)

    x16, b16 = x.bfloat16(), b.bfloat16()

    def calls():                                        # (nothing of torch's that checks for errors)
        q = g.mx4_quantize(x)
        r = g.route(x, 4)
        return (g.mx4_dequantize(q), g.mx4_linear(x, q), g.grouped_linear(x, b, off), g.grouped_linear(x16, b16, off),
                g.grouped_weight_grad(x, x, off), g.route_grad(x, r, grad))

    want = calls()
    hip.hipGetLastError()
    assert hip.hipSetDevice(99) != 0
    try:
        got = calls()
        left = hip.hipGetLastError()
    finally:
        hip.hipGetLastError()
    assert left != 0
    assert all(torch.equal(p, q) for p, q in zip(want, got))
