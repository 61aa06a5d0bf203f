"""orthogonalize against its definition in 64 bits.

Tolerance, of the 2-norm.  bfloat16: the last rounding leaves up to 2^-8 / sqrt(3)
(1.7e-3 measured of any result rounded so: half a step is 2^-9 to 2^-8 of a value); A
and B are held in 11 bits: every step adds an error of 2^-11 |B| over the singular values' size, which the
following steps take on at most unchanged in the directions it falls on: bounded by 5 * 2^-11 = 2.4e-3
on top.  32 bits: 22 bits between the steps and products off by sqrt(k / 16) 2^-24, both multiplied by up
to a^steps = 480 in directions that are small in X: below 480 * 2^-22 = 1.2e-4 in any case;
for inputs without singular values that small (random entries) the factor is their rise, the size of the result
over that of X / |X|, sqrt(order): 1e-5 up to order 1500."""
import pytest
import torch

import dense_gemm_optimisation_fp32_amd as g

pytestmark = pytest.mark.gpu
COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def normal(shape, dtype, seed, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def definition(x, steps=5, coefficients=COEFFICIENTS, scale=1.0):
    x = x.double()
    if x.dim() == 3:
        return torch.stack([definition(v, steps, coefficients, scale) for v in x])
    if x.shape[0] > x.shape[1]:
        return definition(x.t(), steps, coefficients, scale).t()
    size = x.norm()
    if size == 0:
        return x
    x = x / size
    for i in range(steps):
        a, b, c = coefficients if not isinstance(coefficients[0], tuple) else coefficients[i]
        s = x @ x.t()
        x = a * x + (b * s + c * s @ s) @ x
    return scale * x


def room(dtype):
    return 1e-5 if dtype == torch.float32 else 2.0 ** -8 / 3 ** 0.5 + 5 * 2.0 ** -11


def off(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


SHAPES = [(1, 1), (1, 5), (7, 1), (2, 3), (16, 16), (31, 65), (64, 64), (65, 64), (64, 192), (100, 333), (129, 127), (200, 1000),
          (1000, 70), (64, 128), (40, 250), (64, 384), (300, 64), (64, 385), (450, 33), (50, 1024), (1100, 64), (64, 2050), (20, 4200),
          (5000, 64), (65, 66), (128, 64), (90, 128), (128, 128), (129, 130), (100, 400), (512, 128), (128, 513), (70, 1024), (1024, 127),
          (128, 1025), (256, 256), (320, 640), (513, 300), (700, 1100), (1300, 520)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_one_matrix(rows, cols, dtype):
    x = normal((rows, cols), dtype, rows + cols)
    got = g.orthogonalize(x)
    assert got.shape == x.shape and got.dtype == dtype
    assert off(got, definition(x)) <= room(dtype)


# Whole rounds of large tiles, tiles shared by workgroups, both, and sizes that fit none.
LARGE = [(1, 1500, 1600), (1, 2118, 2081), (1, 1027, 5003), (1, 5003, 1027), (3, 1100, 2300), (24, 520, 530), (70, 300, 280), (2, 2048, 2048),
         (5, 1536, 1024)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("batch,rows,cols", LARGE)
def test_large(batch, rows, cols, dtype):
    x = normal((batch, rows, cols), dtype, rows)
    got = g.orthogonalize(x)
    assert torch.equal(got, g.orthogonalize(x))
    for i in {0, batch // 2, batch - 1}:
        assert off(got[i], definition(x[i])) <= room(dtype), i


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("batch,rows,cols", [(0, 8, 8), (1, 20, 30), (5, 64, 96), (33, 70, 40), (6, 64, 500), (40, 120, 100), (5, 100, 700), (3, 300, 200), (9, 260, 513), (70, 256, 256)])
def test_stacks(batch, rows, cols, dtype):
    x = normal((batch, rows, cols), dtype, batch) * torch.exp(3 * normal((batch, 1, 1), torch.float32, 1)).to(dtype)
    got = g.orthogonalize(x, scale=0.5)
    assert got.shape == x.shape
    for i in range(batch):
        assert off(got[i], definition(x[i], scale=0.5)) <= room(dtype), i


def test_singular_values_come_near_one():
    """0.68 to 1.21 is what five steps make of 0.01 to 1 (the scalar map, tabulated here)."""
    u, _ = torch.linalg.qr(normal((96, 96), torch.float32, 1).double().cpu())
    v, _ = torch.linalg.qr(normal((160, 96), torch.float32, 2).double().cpu())
    s = torch.logspace(-1.5, 0, 96, dtype=torch.float64)
    x = (u * s @ v.t()).float().cuda()
    t = s / s.norm()
    for _ in range(5):
        t = COEFFICIENTS[0] * t + COEFFICIENTS[1] * t ** 3 + COEFFICIENTS[2] * t ** 5
    got = g.orthogonalize(x).double().cpu()
    assert ((u.t() @ got @ v).diagonal() - t).abs().max() <= 480 * 2.0 ** -22


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_falling_singular_values(dtype):
    """Few large directions over small noise, where the steps multiply roundings the most."""
    x = (normal((300, 8), torch.float32, 1) @ normal((8, 400), torch.float32, 2) + 1e-3 * normal((300, 400), torch.float32, 3)).to(dtype)
    assert off(g.orthogonalize(x), definition(x)) <= (480 * 2.0 ** -22 if dtype == torch.float32 else room(dtype))


def test_magnitudes_of_any_size():
    """The norm is taken in 64 bits: neither squares nor their sum leave the range."""
    x = normal((40, 60), torch.float32, 5)
    want = definition(x)
    for scale in (1e-30, 1e30, 2.0 ** -126, 2.0 ** 120):
        assert off(g.orthogonalize(x * scale), definition(x * scale)) <= 1e-5
    assert off(g.orthogonalize(x * 2.0 ** 100), want) <= 1e-5
    assert off(g.orthogonalize((x * 1e-41)), definition(x * 1e-41)) <= 1e-5


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(70, 90), (170, 200), (300, 150)])
def test_zeros_and_values_that_are_not_finite(rows, cols, dtype):
    x = normal((4, rows, cols), dtype, 6)
    x[1] = 0
    x[2, 3, 4] = float("inf")
    x[3, 69, 89] = float("nan")
    got = g.orthogonalize(x)
    assert (got[1] == 0).all() and got[2].isnan().any() and got[3].isnan().any()
    assert torch.equal(got[0], g.orthogonalize(x[0]))


def test_steps_and_coefficients():
    x = normal((80, 50), torch.float32, 7)
    assert off(g.orthogonalize(x, steps=1), definition(x, 1)) <= 1e-5
    assert off(g.orthogonalize(x, steps=2), definition(x, 2)) <= 1e-5
    cubic = (1.5, -0.5, 0.0)
    assert off(g.orthogonalize(x, steps=12, coefficients=cubic), definition(x, 12, cubic)) <= 1e-5
    each = ((4.0, -6.0, 2.9), (3.0, -4.0, 2.0), (1.875, -1.25, 0.375))
    assert off(g.orthogonalize(x, steps=3, coefficients=each), definition(x, 3, each)) <= 1e-5
    assert off(g.orthogonalize(x, steps=3, coefficients=[list(c) for c in each], scale=-2.0), definition(x, 3, each, -2.0)) <= 1e-5


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(90, 140), (140, 90), (257, 257)])
def test_strides_out_and_in_place(rows, cols, dtype):
    full = normal((3, rows + 2, cols + 5), dtype, 8)
    x = full[:, 1:1 + rows, 3:3 + cols]
    want = g.orthogonalize(x.contiguous())
    assert torch.equal(g.orthogonalize(x), want)
    turned = g.orthogonalize(x.contiguous().transpose(1, 2).contiguous().transpose(1, 2))
    assert off(turned, want.double()) <= room(dtype)
    out = torch.full((3, rows + 1, cols + 1), 9.0, dtype=dtype, device="cuda")
    g.orthogonalize(x, out=out[:, 1:, 1:])
    assert torch.equal(out[:, 1:, 1:], want) and (out[:, 0] == 9).all() and (out[:, :, 0] == 9).all()
    before = full.clone()
    assert g.orthogonalize(x, out=x) is not None and torch.equal(x, want)
    full[:, 1:1 + rows, 3:3 + cols] = before[:, 1:1 + rows, 3:3 + cols]
    assert torch.equal(full, before)
    one = before[:1, 1:1 + rows, 3:3 + cols].expand(4, rows, cols)          # a matrix read four times
    assert torch.equal(g.orthogonalize(one), want[:1].expand(4, rows, cols))


@pytest.mark.parametrize("rows,cols", [(70, 200), (30, 100), (60, 900), (128, 1000), (200, 300)])
def test_turned_matrices_agree(rows, cols):
    x = normal((rows, cols), torch.float32, 9)
    assert off(g.orthogonalize(x.t().contiguous()).t(), definition(x)) <= 1e-5


@pytest.mark.parametrize("rows,cols", [(40, 60), (40, 350), (40, 800), (100, 100), (100, 800)])
def test_few_rows_zeros_magnitudes_and_strides(rows, cols):
    x = normal((5, rows, cols), torch.float32, 6)
    x[1] = 0
    x[2, 3, 4] = float("inf")
    x[3] *= 1e-30
    x[4] *= 1e30
    got = g.orthogonalize(x)
    assert (got[1] == 0).all() and got[2].isnan().any()
    for i in (0, 3, 4):
        assert off(got[i], definition(x[i])) <= 1e-5
    full = normal((3, rows + 2, cols + 5), torch.bfloat16, 8)
    part = full[:, 1:1 + rows, 3:3 + cols]
    want = g.orthogonalize(part.contiguous())
    before = full.clone()
    g.orthogonalize(part, out=part)
    assert torch.equal(part, want)
    full[:, 1:1 + rows, 3:3 + cols] = before[:, 1:1 + rows, 3:3 + cols]
    assert torch.equal(full, before)
    for steps in (1, 2, 3, 6):
        assert off(g.orthogonalize(x[0], steps=steps), definition(x[0], steps)) <= 1e-5


@pytest.mark.parametrize("batch,rows,cols", [(40, 2048, 2048), (1400, 64, 4096)])
def test_stacks_that_are_worked_on_in_parts(batch, rows, cols):
    """More matrices than 2 GiB of workspace hold: two rounds, also in place."""
    x = normal((batch, rows, cols), torch.float32, 1)
    got = g.orthogonalize(x)
    for i in (0, batch * 3 // 4, batch * 4 // 5, batch - 1):
        assert off(got[i], definition(x[i])) <= 1e-5, i
    g.orthogonalize(x, out=x)
    assert torch.equal(x, got)


@pytest.mark.parametrize("rows,cols", [(100, 100), (300, 200)])
def test_bfloat16_magnitudes(rows, cols):
    x = normal((rows, cols), torch.bfloat16, 2)
    want = g.orthogonalize(x)
    # A power of two gives the same bits, where it is exact: entries of 2^-13 and more times
    # 2^-120 would be subnormal, with fewer bits.
    for power in (-100, -40, 60, 100):
        assert torch.equal(x * 2.0 ** power * 2.0 ** -power, x)
        assert torch.equal(g.orthogonalize(x * 2.0 ** power), want)


def test_refusals():
    x = normal((8, 8), torch.float32, 1)
    for f in ((40.0, 0.0, 0.0), (float("nan"), 0.0, 0.0), (3.0, float("inf"), 0.0), (8.0, 0.0, 0.0)):
        with pytest.raises(g.GemmF32Error):
            g.orthogonalize(x, coefficients=f)              # (8 s grows past 31 in the second step)
    with pytest.raises(ValueError):
        g.orthogonalize(x, steps=0)
    with pytest.raises(ValueError):
        g.orthogonalize(x, steps=65)
    with pytest.raises(ValueError):
        g.orthogonalize(x, steps=10 ** 12)
    with pytest.raises(TypeError):
        g.orthogonalize(x, steps=2.0)
    with pytest.raises(ValueError):
        g.orthogonalize(x, coefficients=(1.0, 2.0))
    with pytest.raises(ValueError):
        g.orthogonalize(x, steps=2, coefficients=((1.0, 0.0, 0.0),) * 3)
    with pytest.raises(ValueError):
        g.orthogonalize(x[0])
    with pytest.raises(ValueError):
        g.orthogonalize(normal((8, 16), torch.float32, 1)[:, ::2])
    with pytest.raises(ValueError):
        g.orthogonalize(x, out=torch.empty((8, 9), device="cuda"))
    with pytest.raises(ValueError):
        g.orthogonalize(x.expand(2, 8, 8), out=torch.empty((8, 8), device="cuda").expand(2, 8, 8))


@pytest.mark.parametrize("rows,cols", [(96, 200), (40, 100), (600, 50), (200, 300), (100, 90)])
def test_captured_replayed_and_on_two_streams(rows, cols):
    x = normal((2, rows, cols), torch.float32, 3)
    want = g.orthogonalize(x)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got += [g.orthogonalize(x) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(v, want) for v in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = g.orthogonalize(x)
    for seed in range(3):
        x.copy_(normal((2, rows, cols), torch.float32, 30 + seed))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, g.orthogonalize(x))
