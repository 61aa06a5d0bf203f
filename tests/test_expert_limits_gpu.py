"""The expert-layer operators far out in their ranges, on the GPU: rows far
apart, and far from the first.

Tolerance of a 32-bit product, per element: the library's bar 1e-5 S + 1e-6, S
the sum of the terms' magnitudes."""
import pytest
import torch

import dense_gemm_optimisation_fp32_amd as g

pytestmark = pytest.mark.gpu

DEV = "cuda"


def normal(shape, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return torch.randn(shape, generator=gen, device=DEV)


def close(y, a, b):
    ref, s = a.double() @ b.double(), a.double().abs() @ b.double().abs()
    assert ((y.double() - ref).abs() <= 1e-5 * s + 1e-6).all()


def offsets(*ends):
    return torch.tensor(ends, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("rows,k,n", [(600, 5, 7), (600, 1500, 1500), (600, 1500, 1320), (1300, 1500, 1500)])
def test_f32_weight_grad_over_rows_far_apart(rows, k, n):
    """Rows of A almost 8 MiB apart: the contraction is taken in runs of 255
    rows, whose offsets fit 31 bits.  The cases take the kernel's four tiles."""
    apart = (1 << 21) - 1
    a = torch.empty(rows * apart, device=DEV).as_strided((rows, k), (apart, 1))
    a.copy_(normal((rows, k), 1))
    grad = normal((rows, n), 2)
    out = g.grouped_weight_grad(a, grad, offsets(0, 10, rows))
    close(out[0], a[:10].t().contiguous(), grad[:10])
    close(out[1], a[10:].t().contiguous(), grad[10:])


def test_f32_weight_grad_of_an_expert_whose_rows_begin_far_out():
    """One column, rows from 1.9e9 on: the row that a run begins at, plus the
    rows of a run, passes 2^31."""
    first, rows = 1_900_000_000, 1000
    a = torch.empty((first + rows, 1), device=DEV)
    grad = torch.empty((first + rows, 1), device=DEV)
    a[first:], grad[first:] = normal((rows, 1), 3), normal((rows, 1), 4)
    out = g.grouped_weight_grad(a, grad, offsets(first, first + rows))
    close(out[0], a[first:].t(), grad[first:])
