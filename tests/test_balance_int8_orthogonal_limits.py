"""Limits of 8-bit quantisation and orthogonalising that go by what the kernels count in
32 bits or hold in half precision (no GPU compute): beyond them a call is refused before
it touches a device, within them it reaches the device check."""
import pytest
import torch

import dense_gemm_optimisation_fp32_amd as g
from dense_gemm_optimisation_fp32_amd import expert_ops as x

OK = 0x10000            # a well aligned address that is never followed
BAD = g.GEMM_F32_ERR_INVALID_VALUE
ACCEPTED = g.GEMM_F32_ERR_NO_DEVICE
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not real")


def wraps(k, step):
    """Whether columns counted in `step` pass 2^31 - 1 before the loop over them ends."""
    padded = (k + 15) // 16 * 16
    return (padded + step - 1) // step * step > 2 ** 31 - 1


@pytest.mark.parametrize("k,accepted", [(2 ** 31 - 2049, True), (2 ** 31 - 2047, False), (2 ** 31 - 1500, False), (2 ** 31 - 1, False)])
@pytest.mark.parametrize("layout", [0, 1])
def test_columns_of_a_quantised_matrix(k, accepted, layout):
    """Rows are taken in pieces of 2048 columns."""
    assert accepted or wraps(k, 2048)
    assert not accepted or not wraps(k, 2048)
    status = x._functions()["expert_int8_quantize"](0, 2, k, OK, layout, 2 if layout else k, OK, OK, None)
    assert status == (ACCEPTED if accepted else BAD)


def status_of(f, steps):
    """Of two matrices of 180 x 200 with these coefficients in every step."""
    import ctypes

    values = (ctypes.c_float * (3 * steps))(*(f * steps))
    return x._functions()["expert_orthogonalize"](0, 2, 180, 200, OK, 200, 36000, steps, ctypes.addressof(values), 1.0, OK, 200,
                                                  36000, OK, 1 << 31, None)


@pytest.mark.parametrize("c", [0.0, 1e-10, 1e-14, 1e-17, 1e-20, 1e-30, -1e-14, -1e-17, -1e-20, -1e-30])
@pytest.mark.parametrize("a,b,steps,accepted", [(29.0, -29.0, 1, True), (29.0, -29.0, 2, False), (8.0, -8.0, 3, False), (2.0, -1.0, 6, True),
                                                (-29.0, 29.0, 2, False), (1.5, -0.5, 40, True)])
def test_coefficients_with_a_small_last_one(a, b, c, steps, accepted):
    """29 s - 29 s^3 rises to 11.2 at s = 0.58 and is 0 at 1: two steps leave the range of a
    plane, and a term of 1e-20 s^5 more does not change that."""
    assert status_of((a, b, c), steps) == (ACCEPTED if accepted else BAD)


@pytest.mark.parametrize("seed", range(8))
def test_coefficients_against_a_scan(seed):
    """Largest entries by a scan of 20001 singular values: a call is accepted up to 30.5 and refused from
    31.5 on (the scan misses a maximum by less: its step is 5e-5 of the range, the slopes there below 200)."""
    import random

    rng = random.Random(seed)
    for _ in range(60):
        f = [rng.uniform(-9, 9), rng.uniform(-20, 20), rng.uniform(-20, 20) * 10.0 ** -rng.choice((0, 0, 1, 4, 9, 13, 16, 25))]
        f = [torch.tensor(v).item() for v in f]
        top, most, ends = 1.0, 0.0, []
        for i in range(3):
            s = torch.linspace(0.0, 1.0, 20001, dtype=torch.float64) * top
            u = s * s
            q = (f[0] + f[1] * u + f[2] * u * u).abs()
            ends.append(max(most, top * top, q.max().item()))
            top = (s * q).max().item()
            most = max(ends[-1], top)
            if most > 100:
                break
        for steps, size in enumerate(ends, 1):
            if size < 30.5 or size > 31.5:
                assert status_of(tuple(f), steps) == (ACCEPTED if size < 30.5 else BAD), (f, steps, size)
