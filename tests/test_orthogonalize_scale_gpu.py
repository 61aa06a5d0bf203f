"""orthogonalize with scales from the smallest to the largest that leave the result in the
range of 32 bits: the scale is one more rounding, at any size.

Tolerance: as without a scale, 1e-5 in the 2-norm (random entries, 32 bits)."""
import pytest
import torch

import dense_gemm_optimisation_fp32_amd as g

pytestmark = pytest.mark.gpu


# One strip, several strips, tiles, with either side longer.
@pytest.mark.parametrize("rows,cols", [(40, 60), (60, 40), (60, 900), (900, 60), (170, 200), (200, 170), (700, 900), (900, 700)])
@pytest.mark.parametrize("steps", [1, 5])
def test_scales_of_any_size(rows, cols, steps):
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn((rows, cols), generator=gen, device="cuda")
    want = g.orthogonalize(x, steps=steps)
    for scale in (3e-35, 1e-33, -2e-30, 3e30, 1e37):
        # (Entries below 1e-38 are subnormal, off by 7e-46: nothing beside a norm of 1e-35.)
        got = g.orthogonalize(x, steps=steps, scale=scale).double()
        exact = want.double() * scale
        assert got.isfinite().all()
        assert ((got - exact).norm() / exact.norm()).item() <= 1e-5, scale


def test_scales_that_are_powers_of_two_give_the_same_bits():
    gen = torch.Generator(device="cuda").manual_seed(1)
    for shape in ((40, 60), (60, 900), (170, 200), (200, 170)):
        x = torch.randn(shape, generator=gen, device="cuda")
        want = g.orthogonalize(x)
        for power in (-80, -1, 60, 110):
            assert torch.equal(g.orthogonalize(x, scale=2.0 ** power), want * 2.0 ** power)
