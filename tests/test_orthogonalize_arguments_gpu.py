"""orthogonalize's coefficients of any number type, and `out` of matrices with unit stride
along either axis."""
import numpy as np
import pytest
import torch

import dense_gemm_optimisation_fp32_amd as g

pytestmark = pytest.mark.gpu
TRIPLE = (3.4445, -4.7750, 2.0315)


def normal(shape, seed):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def test_numbers_of_any_type():
    x = normal((40, 60), 1)
    want = g.orthogonalize(x)
    for given in (np.array(TRIPLE, dtype=np.float32), torch.tensor(TRIPLE), [TRIPLE] * 5, np.array([TRIPLE] * 5, dtype=np.float32),
                  [torch.tensor(TRIPLE)] * 5):
        assert torch.equal(g.orthogonalize(x, coefficients=given), want)
    with pytest.raises(ValueError):
        g.orthogonalize(x, steps=4, coefficients=[TRIPLE] * 5)


@pytest.mark.parametrize("shape", [(40, 60), (3, 200, 300), (2, 60, 40)])
def test_out_of_a_turned_matrix(shape):
    x = normal(shape, 2).transpose(-1, -2)
    want = g.orthogonalize(x)
    assert want.stride() == x.stride()
    out = torch.empty(shape, device="cuda").transpose(-1, -2)
    assert g.orthogonalize(x, out=out) is out and torch.equal(out, want)
    for bad in (torch.empty(x.shape, device="cuda"), torch.empty(shape, device="cuda")):
        with pytest.raises(ValueError, match="out"):
            g.orthogonalize(x, out=bad)
    with pytest.raises(ValueError, match="out"):
        g.orthogonalize(x.contiguous(), out=out)
    assert g.orthogonalize(x, out=x) is x and torch.equal(x, want)
