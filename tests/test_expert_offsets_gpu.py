"""Offsets that are not sorted or point outside, on the GPU: the products write
inside their result and nowhere else.  The result is a part of a larger tensor
whose other elements have to stay as they are; what is written inside is not
looked at."""
import pytest
import torch

import dense_gemm_optimisation_fp32_amd as g

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DEV = "cuda"
KEPT = 7.0


def normal(shape, dtype, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return torch.randn(shape, generator=gen, device=DEV).to(dtype)


def wrong_offsets(m, groups):
    """Lists of groups + 1 ends: far outside, falling, all before the first row,
    every expert with every row."""
    lists = [[(0, 5 * m, -3, 10 * m)[i % 4] for i in range(groups + 1)],
             [m - m * i // groups if i % 2 else m * i // (2 * groups) for i in range(groups + 1)],
             [-5] * (groups + 1),
             [(0, m)[i % 2] for i in range(groups + 1)],
             [(-2 ** 31, 2 ** 31 - 1)[i % 2] for i in range(groups + 1)]]
    return [torch.tensor(x, dtype=torch.int32, device=DEV) for x in lists]


def inside(shape, dtype):
    """A result of `shape` with rows and columns around it (and matrices, of three
    dimensions), and the whole."""
    margins = [3] * (len(shape) - 1) + [8]                    # (16 bytes: aligned results stay aligned)
    whole = torch.full([n + 2 * s for n, s in zip(shape, margins)], KEPT, dtype=dtype, device=DEV)
    part = whole
    for d, (n, s) in enumerate(zip(shape, margins)):
        part = part.narrow(d, s, n)
    return part, whole


def nothing_outside(part, whole, what):
    torch.cuda.synchronize()
    part.fill_(KEPT)
    assert (whole == KEPT).all(), what


# Rows, experts, n, k: each of the kernels (few rows an expert, few tiles, 64 and
# 128 rows a tile, the pipeline of 256), and rows of odd length.
SIZES = [(60, 4, 64, 64), (60, 4, 67, 65), (100, 4, 64, 64), (100, 4, 131, 65), (1000, 3, 200, 96), (600, 2, 8200, 40),
         (1200, 40, 4104, 40), (300, 2, 16400, 33), (1000, 3, 13304, 64), (1500, 3, 13303, 70)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("m,groups,n,k", SIZES)
def test_grouped_linear(dtype, layout, m, groups, n, k):
    a, b = normal((m, k), dtype, 1), normal((groups, k, n) if layout == "row" else (groups, n, k), dtype, 2)
    for i, off in enumerate(wrong_offsets(m, groups)):
        out, whole = inside((m, n), dtype)
        g.grouped_linear(a, b if layout == "row" else b.transpose(1, 2), off, out=out)
        nothing_outside(out, whole, f"offsets {i}")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,groups,n,k", [(60, 4, 64, 64), (60, 4, 67, 65), (100, 3, 600, 700), (300, 2, 1203, 1305),
                                          (1500, 3, 2560, 2560), (1500, 3, 2562, 2054)])
def test_grouped_weight_grad(dtype, m, groups, n, k):
    a, grad = normal((m, k), dtype, 3), normal((m, n), dtype, 4)
    for i, off in enumerate(wrong_offsets(m, groups)):
        out, whole = inside((groups, k, n), dtype)
        g.grouped_weight_grad(a, grad, off, out=out)
        nothing_outside(out, whole, f"offsets {i}")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,groups,n,k", SIZES)
def test_mx4_linear(dtype, m, groups, n, k):
    q = g.mx4_quantize(normal((groups * n, k), F32, 5))
    kb = q.scales.shape[0]
    w = g.Mx4Tensor(q.codes.view(groups, n, -1), q.scales.view(kb, groups, n, 4).transpose(0, 1).contiguous(), k)
    x = normal((m, k), dtype, 6)
    for i, off in enumerate(wrong_offsets(m, groups)):
        out, whole = inside((m, n), dtype)
        g.mx4_linear(x, w, offsets=off, out=out)
        nothing_outside(out, whole, f"offsets {i}")


def test_the_check_finds_a_write_outside():
    part, whole = inside((4, 16), F32)
    whole[2, 20] = 0
    with pytest.raises(AssertionError, match="planted"):
        nothing_outside(part, whole, "planted")
