"""8-bit quantisation and products on the GPU against a plain implementation.

Codes and scales are defined step by step in 32 bits: equal.  The sums of a
product are whole numbers, exact; then four roundings of 2^-24 (to 32 bits, two
scales, bias) and, with an activation, GELU's approximation (1.5e-7 absolute in
erf, 8 roundings): room of 4 * 2^-24 of |y| and of |bias|, for GELU 16 * 2^-24 of
|y| and |bias| and 1e-7 |y| more; then half a step of the result's type."""
import pytest
import torch

import dense_gemm_optimisation_fp32_amd as g

pytestmark = pytest.mark.gpu
INF = float("inf")


def normal(shape, dtype, seed, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def quantised(x):
    """Codes and scales of the rows of x, each step in 32 bits (numpy's divisions are IEEE's)."""
    import numpy as np

    v = x.float().cpu().numpy()
    with np.errstate(all="ignore"):
        top = np.abs(v).max(1)
        bad = ~np.isfinite(v).all(1)
        none = top < np.float32(2.0 ** -119)
        inverse = np.where(bad | none, np.float32(0), np.float32(127) / np.where(none, np.float32(1), top))
        codes = np.where(bad[:, None], np.float32(0), np.rint(v * inverse[:, None].astype(np.float32)))
        scales = np.where(bad, np.float32("nan"), np.where(none, np.float32(0), top / np.float32(127)))
    return torch.from_numpy(codes.astype("int8")), torch.from_numpy(scales.astype("float32"))


def check_codes(x):
    q = g.int8_quantize(x)
    r, k = x.shape
    codes, scales = quantised(x)
    assert q.codes.shape == (r, (k + 15) // 16 * 16) and tuple(q.shape) == (r, k)
    assert torch.equal(q.codes[:, :k].cpu(), codes)
    assert (q.codes[:, k:] == 0).all()
    assert torch.equal(q.scales.cpu().view(torch.int32) & 0x7fc00000, scales.view(torch.int32) & 0x7fc00000)
    finite = scales == scales
    assert torch.equal(q.scales.cpu()[finite], scales[finite])
    return q, codes, scales


SHAPES = [(1, 1), (1, 16), (3, 17), (5, 70), (130, 128), (7, 513), (66, 2048), (9, 2049), (4, 2300), (3, 8192), (2, 8200), (2, 20001)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("r,k", SHAPES)
def test_quantize_and_back(r, k, dtype):
    x = normal((r, k), dtype, r + k) * torch.exp(normal((r, 1), torch.float32, r)).to(dtype)
    for v in (x, normal((k, r), dtype, k).t(), normal((r, k + 5), dtype, 3)[:, 2:2 + k]):
        q, codes, scales = check_codes(v)
        for to in (torch.float32, torch.bfloat16):
            want = (codes.float() * scales.unsqueeze(1)).to(to)
            assert torch.equal(g.int8_dequantize(q, to).cpu(), want)
    out = torch.full((r, k + 3), 7.0, device="cuda")
    g.int8_dequantize(q, out=out[:, 1:1 + k])
    assert (out[:, 0] == 7).all() and (out[:, 1 + k:] == 7).all()


@pytest.mark.parametrize("turned", [False, True])
def test_rows_of_zeros_infinities_and_extremes(turned):
    x = normal((12, 100), torch.float32, 5)
    x[1] = 0
    x[2, 7] = INF
    x[3, 99] = float("nan")
    x[4] *= 1e-40                              # below the normal numbers
    x[5] *= 3e37
    x[6] = 2.0 ** -119
    x[7] = 2.0 ** -119 * (1 - 2.0 ** -24)      # just below the least
    x[8] = -0.0
    x[9] = torch.arange(100, device="cuda") - 127.0 / 2    # ties
    x[10, :] = 127.0
    x[10, 1:] = torch.arange(99, device="cuda") + 0.5      # ties to even
    if turned:
        x = x.t().contiguous().t()
    q, _, _ = check_codes(x)
    assert q.scales[2].isnan() and q.scales[3].isnan() and (q.codes[2] == 0).all()
    assert q.scales[7] == 0 and q.scales[4] == 0 and q.scales[6] > 0
    y = g.int8_dequantize(q)
    assert y[2].isnan().all() and (y[1] == 0).all()


def test_no_rows():
    q = g.int8_quantize(torch.empty((0, 40), device="cuda"))
    assert q.codes.shape == (0, 48) and g.int8_dequantize(q).shape == (0, 40)
    assert g.int8_linear(torch.empty((0, 40), device="cuda"), g.int8_quantize(normal((5, 40), torch.float32, 1))).shape == (0, 5)


def weights(groups, n, k, seed):
    """Codes with every value from -127 to 127, scales of different magnitude, on the GPU."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    shape = (groups, n) if groups else (n,)
    codes = torch.zeros((*shape, (k + 15) // 16 * 16), dtype=torch.int8, device="cuda")
    codes[..., :k] = torch.randint(-127, 128, (*shape, k), generator=gen, device="cuda", dtype=torch.int8)
    scales = torch.exp(torch.randn(shape, generator=gen, device="cuda")) / 127 * k ** -0.5
    return g.Int8Tensor(codes, scales, k)


def expected(x, w, offsets, bias, act):
    codes, scales = quantised(x)
    m, n, k = x.shape[0], w.shape[-2], w.k
    y, size = torch.zeros((m, n), dtype=torch.float64), torch.zeros((m, n), dtype=torch.float64)
    ends = [0, m] if offsets is None else offsets.tolist()
    for e in range(len(ends) - 1):
        lo, hi = ends[e], ends[e + 1]
        wc, ws = (w.codes, w.scales) if offsets is None else (w.codes[e], w.scales[e])
        v = codes[lo:hi].double() @ wc[:, :k].double().cpu().t() * scales[lo:hi].double().unsqueeze(1) * ws.double().cpu()
        much = v.abs()
        if bias is not None:
            b = (bias if bias.dim() == 1 else bias[e]).double().cpu()
            v, much = v + b, much + b.abs()
        if act == "relu":
            v = torch.relu(v)
        elif act == "gelu":
            v = v * torch.special.ndtr(v)
        y[lo:hi], size[lo:hi] = v, much
    return y, size


def check_product(x, w, offsets=None, bias=None, act=None, out=None):
    got = g.int8_linear(x, w, offsets=offsets, bias=bias, activation=act, out=out)
    want, size = expected(x, w, offsets, bias, act)
    room = (16 * 2.0 ** -24 + 1e-7 if act == "gelu" else 4 * 2.0 ** -24) * size + torch.finfo(x.dtype).eps / 2 * want.abs()
    off = (got.double().cpu() - want).abs()
    assert (off <= room * 1.001).all(), (off / room.clamp(min=1e-300)).max().item()
    return got


# Rows, columns and contractions around tiles, strips, slabs and instructions.
DENSE = [(1, 1, 1), (1, 17, 16), (4, 130, 100), (16, 33, 257), (17, 64, 128), (5, 4100, 300), (33, 300, 513), (64, 1000, 640),
         (65, 129, 2049), (200, 520, 200), (257, 2050, 128), (300, 1024, 1023), (1000, 1536, 384), (770, 8200, 130), (2050, 2304, 255),
         (2050, 8201, 140), (2100, 8192, 300)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n,k", DENSE)
def test_linear(m, n, k, dtype):
    x, w = normal((m, k), dtype, m + n), weights(0, n, k, k)
    act = (None, "relu", "gelu")[(m + k) % 3]
    check_product(x, w, bias=normal((n,), torch.float32, 7) if n % 2 else None, act=act)


def offsets_of(sizes):
    return torch.tensor([0, *torch.tensor(sizes).cumsum(0).tolist()], dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes,n,k", [
    ([2, 0, 1, 0], 70, 40), ([0, 0, 3], 33, 130), ([16, 17, 15, 1, 0, 31], 200, 260), ([100, 0, 1, 37, 64, 65], 300, 200),
    ([300, 260, 0, 250, 1], 600, 384), ([129] * 20, 513, 100), ([700, 400, 600], 4100, 260), ([900, 1101, 0, 700, 1], 8200, 260), ([0] * 70 + [5] + [0] * 9, 48, 33),
    ([0] * 30 + [41] + [0] * 20 + [1], 100, 700), ([1, 2, 2, 3], 4500, 1500), ([8, 9, 1, 16] * 15, 600, 300)])
def test_linear_by_expert(sizes, n, k, dtype):
    m = sum(sizes)
    x, w, off = normal((m, k), dtype, m), weights(len(sizes), n, k, n), offsets_of(sizes)
    check_product(x, w, off, normal((len(sizes), n), torch.float32, 3), "gelu" if n % 2 else None)


@pytest.mark.parametrize("rows,n", [(6, 40), (90, 200), (900, 1100), (1200, 6000)])
def test_rows_of_no_expert_are_zero(rows, n):
    """Before the first expert's and after the last one's, also with an infinity in them."""
    x, w = normal((rows, 96), torch.float32, 5), weights(2, n, 96, 5)
    x[0] = INF
    lo, mid, hi = rows // 6, rows // 2, rows - rows // 5
    got = g.int8_linear(x, w, offsets=torch.tensor([lo, mid, hi], dtype=torch.int32, device="cuda"),
                        bias=torch.ones((2, n), device="cuda"), activation="gelu")
    assert (got[:lo] == 0).all() and (got[hi:] == 0).all() and (got[lo:hi] != 0).any()


@pytest.mark.parametrize("m,n,k", [(3, 100, 300), (40, 500, 100), (600, 700, 129)])
def test_rows_that_are_not_finite_stay_their_own(m, n, k):
    x, w = normal((m, k), torch.float32, 9), weights(0, n, k, 9)
    clean = g.int8_linear(x, w)
    x[m // 2, k - 1] = float("nan")
    x[0, 0] = -INF
    got = g.int8_linear(x, w)
    assert got[m // 2].isnan().all() and got[0].isnan().all()
    others = [i for i in range(m) if i not in (0, m // 2)]
    assert torch.equal(got[others], clean[others])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides_and_out(dtype):
    x = normal((50, 300), dtype, 4)[:, 7:207]
    w = weights(0, 77, 200, 4)
    out = torch.full((50, 100), 5.0, dtype=dtype, device="cuda")
    got = check_product(x, w, out=out[:, 11:88])
    assert got.data_ptr() == out[:, 11:].data_ptr()
    assert (out[:, :11] == 5).all() and (out[:, 88:] == 5).all()
    check_product(normal((200, 50), dtype, 6).t().contiguous()[::2], w)


def test_largest_sums_do_not_wrap():
    """The longest contraction, all codes 127: 127 * 127 * 131072 is below 2^31."""
    k = 131072
    x = torch.ones((2, k), device="cuda")
    w = g.Int8Tensor(torch.full((3, k), 127, dtype=torch.int8, device="cuda"), torch.ones(3, device="cuda"), k)
    got = g.int8_linear(x, w).double().cpu()
    want = 127.0 * k
    assert ((got - want).abs() <= want * 4 * 2.0 ** -24).all()
    with pytest.raises(g.GemmF32Error):
        g.int8_linear(torch.ones((2, k + 1), device="cuda"), weights(0, 3, k + 1, 1))


def test_wrong_offsets_write_inside():
    x, w = normal((40, 64), torch.float32, 5), weights(3, 50, 64, 5)
    for bad in ([0, 30, 10, 40], [-5, 10, 20, 90], [40, 0, 40, 0]):
        out = torch.zeros((60, 50), device="cuda")
        g.int8_linear(x, w, offsets=torch.tensor(bad, dtype=torch.int32, device="cuda"), out=out[10:50])
        assert (out[:10] == 0).all() and (out[50:] == 0).all()


def test_same_bits_each_time_on_two_streams_and_replayed():
    x, w = normal((130, 1000), torch.bfloat16, 5), weights(0, 1500, 1000, 5)
    want = g.int8_linear(x, w, activation="gelu")
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for s in streams:
        with torch.cuda.stream(s):
            got += [g.int8_linear(x, w, activation="gelu") for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(v, want) for v in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = g.int8_linear(x, w, activation="gelu")
        few = g.int8_linear(x[:3], w)
    for seed in range(3):
        x.copy_(normal((130, 1000), torch.bfloat16, 20 + seed))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, g.int8_linear(x, w, activation="gelu")) and torch.equal(few, g.int8_linear(x[:3], w))


def test_refusals():
    x, w = normal((6, 40), torch.float32, 1), weights(0, 5, 40, 1)
    many, off = weights(3, 5, 40, 1), offsets_of([2, 2, 2])
    for bad in (dict(w=weights(0, 5, 41, 1)), dict(w=many), dict(offsets=off), dict(w=many, offsets=off[:3]),
                dict(w=many, offsets=off.long()), dict(bias=torch.zeros(4, device="cuda")), dict(bias=torch.zeros(5)),
                dict(out=torch.empty((6, 6), device="cuda")), dict(out=torch.empty((6, 5), device="cuda").bfloat16()),
                dict(w=g.Int8Tensor(w.codes.cpu(), w.scales.cpu(), 40))):
        with pytest.raises(ValueError):
            g.int8_linear(**{"x": x, "w": w, **bad})
    with pytest.raises(TypeError):
        g.int8_linear(x.half(), w)
    with pytest.raises(ValueError):
        g.int8_linear(x[:, ::2], weights(0, 5, 20, 1))
    with pytest.raises(ValueError):
        g.int8_quantize(normal((4, 6, 8), torch.float32, 1))
    with pytest.raises(ValueError):
        g.int8_quantize(normal((8, 16), torch.float32, 1)[::2, ::2])
    with pytest.raises(ValueError):
        g.int8_dequantize(many)
    # Codes that do not begin at 16 bytes: refused by the library.
    base = torch.zeros(5 * 48 + 4, dtype=torch.int8, device="cuda")
    with pytest.raises(g.GemmF32Error):
        g.int8_linear(x, g.Int8Tensor(base[4:].view(5, 48), torch.ones(5, device="cuda"), 40))


@pytest.mark.parametrize("offset", [1, 2, 3])
def test_rows_at_any_address(offset):
    """x and the result at addresses of their type's alignment, rows of odd length."""
    base = normal((70 * 333 + 8,), torch.bfloat16, 3)
    x = base[offset:offset + 70 * 333].view(70, 333)
    out = torch.empty(70 * 77 + 8, dtype=torch.bfloat16, device="cuda")[offset:offset + 70 * 77].view(70, 77)
    check_product(x, weights(0, 77, 333, 4), out=out)
    check_product(x[:3], weights(0, 77, 333, 5), out=out[:3])
    check_codes(x)
