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


def test_weight_gradients_that_overlap_are_refused():
    a, off = torch.randn((8, 32), device=DEV), torch.tensor([0, 3, 5, 6, 8], dtype=torch.int32, device=DEV)
    grad = torch.randn((8, 16), device=DEV)
    with pytest.raises(ValueError, match="overlapping"):
        g.grouped_weight_grad(a, grad, off, out=torch.empty((1, 32, 16), device=DEV).expand(4, 32, 16))
    with pytest.raises(ValueError, match="overlapping"):
        g.grouped_weight_grad(a, grad, off, out=torch.empty(4096, device=DEV).as_strided((4, 32, 16), (500, 16, 1)))
    want = g.grouped_weight_grad(a, grad, off)
    for out in (torch.empty((32, 4, 16), device=DEV).transpose(0, 1), torch.empty((4, 33, 17), device=DEV)[:, :32, :16]):
        assert torch.equal(g.grouped_weight_grad(a, grad, off, out=out), want)


@pytest.mark.parametrize("offsets", [[], [0]])
def test_weight_gradients_of_no_expert_are_refused(offsets):
    """Two offsets are the least: ValueError, as for every wrong argument."""
    a, off = torch.randn((8, 32), device=DEV), torch.tensor(offsets, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="offsets"):
        g.grouped_weight_grad(a, a, off)
