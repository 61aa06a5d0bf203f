"""orthogonalize's arguments as far as they are seen without a GPU: a CPU matrix is refused
last, so whatever else is wrong is named before it."""
import numpy as np
import pytest
import torch

import dense_gemm_optimisation_fp32_amd as g

TRIPLE = (3.4445, -4.7750, 2.0315)


@pytest.mark.parametrize("coefficients", [
    TRIPLE, list(TRIPLE), np.array(TRIPLE), np.array(TRIPLE, dtype=np.float32), np.array(TRIPLE, dtype=np.float16),
    tuple(np.float32(v) for v in TRIPLE), (np.float32(3.0), -4, 2.0), (3, -4, 2), [TRIPLE] * 5, np.array([TRIPLE] * 5, dtype=np.float32),
    tuple(np.array(TRIPLE, dtype=np.float32) for _ in range(5)), torch.tensor(TRIPLE), torch.tensor([TRIPLE] * 5), [torch.tensor(TRIPLE)] * 5])
def test_numbers_of_any_type(coefficients):
    with pytest.raises(ValueError, match="on a GPU"):
        g.orthogonalize(torch.zeros(4, 8), coefficients=coefficients)


@pytest.mark.parametrize("coefficients", [("a", "b", "c"), 3.0, None, (None, None, None), ((1.0, "x", 2.0),) * 5, [object()] * 3])
def test_what_is_no_number(coefficients):
    with pytest.raises(TypeError, match="coefficients"):
        g.orthogonalize(torch.zeros(4, 8), coefficients=coefficients)


@pytest.mark.parametrize("shape", [(4, 8), (3, 4, 8)])
def test_out_of_a_turned_matrix(shape):
    """x with unit stride along its columns takes such an out, and the message says so."""
    x = torch.zeros(shape).transpose(-1, -2)
    like = torch.zeros(shape).transpose(-1, -2)
    with pytest.raises(ValueError, match="on a GPU"):
        g.orthogonalize(x, out=like)
    with pytest.raises(ValueError, match="out .* same axis as x"):
        g.orthogonalize(x, out=like.contiguous())
    with pytest.raises(ValueError, match="out .*8, 4"):
        g.orthogonalize(x, out=torch.zeros(shape))
    with pytest.raises(TypeError, match="out"):
        g.orthogonalize(x, out=[[0.0] * 4] * 8)
