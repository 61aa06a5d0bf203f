"""orthogonalize of bfloat16 matrices is rounded once: what is held between the steps
is as precise as for 32-bit ones.

Tolerance.  The result is round(y + d): y by the definition in 64 bits, d what the steps
lose, at most 1e-5 of y in the 2-norm, as of 32-bit matrices with random entries up to
order 1500 (22 bits between the steps, 2^-22, times the rise of X, sqrt(order)).  The
rounding is off by half a step of y + d at most, which is y's, or twice that where d takes
y over a power of two; there y + d is within |d| of that power, and rounds to it.  So what an
entry is off beyond half a step of y is at most 2 |d|: 2e-5 of y in the 2-norm, all
entries together."""
import pytest
import torch

import dense_gemm_optimisation_fp32_amd as g

pytestmark = pytest.mark.gpu
COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def definition(x, steps):
    x = x.double()
    if x.shape[0] > x.shape[1]:
        return definition(x.t().contiguous(), steps).t()
    x = x / x.norm()
    for _ in range(steps):
        a, b, c = COEFFICIENTS
        s = x @ x.t()
        x = a * x + (b * s + c * s @ s) @ x
    return x


def beyond_half_a_step(got, want):
    """2-norm of what the entries are off beyond half a step of bfloat16 (8 bits), of want's."""
    half = torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=1e-300))) - 8)
    return (((got.double() - want).abs() - half).clamp(min=0).norm() / want.norm()).item()


# One strip, several, tiles of every kind with whole rounds and shared ones, either side longer.
SHAPES = [(1, 64, 192), (1, 100, 400), (1, 128, 1000), (1, 129, 130), (1, 300, 1000), (1, 700, 300), (1, 1088, 1300), (1, 1500, 1600),
          (1, 1027, 5003), (1, 5003, 1027), (24, 520, 530), (5, 1024, 1500)]


@pytest.mark.parametrize("steps", [1, 2, 5])
@pytest.mark.parametrize("batch,rows,cols", SHAPES)
def test_rounded_once(batch, rows, cols, steps):
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    x = torch.randn((batch, rows, cols), generator=gen, device="cuda").bfloat16()
    got = g.orthogonalize(x, steps=steps)
    for i in {0, batch - 1}:
        assert beyond_half_a_step(got[i], definition(x[i], steps)) <= 2e-5, i
