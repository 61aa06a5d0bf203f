"""The expert-layer operators far out in their ranges, on the GPU: rows far
apart, and far from the first.

Tolerance of a 32-bit product, per element: the library's bar 1e-5 S + 1e-6, S
the sum of the terms' magnitudes; products of bfloat16 or 4-bit values are
exact in 32 bits, so their sums meet the same bar, and a bfloat16 result adds
its rounding, 2^-8 of the value."""
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
    bar = 1e-5 * s + 1e-6
    if y.dtype == torch.bfloat16:
        bar = bar * (1 + 2 ** -8) + 2 ** -8 * ref.abs()
    assert ((y.double() - ref).abs() <= bar).all()


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


def far_apart(shape, dtype):
    """A matrix whose rows are almost 8 MiB apart: its end is gigabytes from its
    beginning."""
    apart = (8 << 20) // dtype.itemsize - 8
    return torch.empty(shape[0] * apart, dtype=dtype, device=DEV).as_strided(shape, (apart, 1))


# Rows, n, k: few rows an expert; few tiles; 64 and 128 rows a tile; the pipeline of
# 256 (bfloat16 and 4 bits).
FAR = [(20, 200, 96), (300, 200, 96), (600, 8200, 40), (1200, 13304, 64)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("m,n,k", FAR)
def test_grouped_linear_with_rows_far_apart(dtype, layout, m, n, k):
    a, out = far_apart((m, k), dtype), far_apart((m, n), dtype)
    a.copy_(normal((m, k), 5))
    b = normal((2, k, n) if layout == "row" else (2, n, k), 6).to(dtype)
    b = b if layout == "row" else b.transpose(1, 2)
    half = m // 2 - 3
    g.grouped_linear(a, b, offsets(0, half, m), out=out)
    close(out[:half], a[:half].contiguous(), b[0].contiguous())
    close(out[half:], a[half:].contiguous(), b[1].contiguous())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n,k", FAR)
def test_mx4_linear_with_rows_far_apart(dtype, m, n, k):
    x, out = far_apart((m, k), dtype), far_apart((m, n), dtype)
    x.copy_(normal((m, k), 7))
    w = g.mx4_quantize(normal((n, k), 8))
    g.mx4_linear(x, w, out=out)
    close(out, g.mx4_dequantize(g.mx4_quantize(x)), g.mx4_dequantize(w).t())


@pytest.mark.parametrize("rows,k,n", [(300, 200, 96), (700, 2100, 2104)])
def test_bf16_weight_grad_with_rows_far_apart(rows, k, n):
    a, grad = far_apart((rows, k), torch.bfloat16), far_apart((rows, n), torch.bfloat16)
    a.copy_(normal((rows, k), 9))
    grad.copy_(normal((rows, n), 10))
    out = far_apart((k, n), torch.bfloat16).unsqueeze(0)
    g.grouped_weight_grad(a, grad, offsets(0, rows), out=out)
    close(out[0], a.t().contiguous(), grad.contiguous())
