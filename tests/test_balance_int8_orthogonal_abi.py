"""Host-side checks of balanced routing, 8-bit products and orthogonalising (no GPU
compute): every entry point refuses bad arguments before it touches a device or an
operand, and the Python layer names what is wrong."""
import ctypes

import pytest
import torch

import dense_gemm_optimisation_fp32_amd as g
from dense_gemm_optimisation_fp32_amd import expert_ops as x

OK = 0x10000            # a well aligned address that is never followed
BAD = g.GEMM_F32_ERR_INVALID_VALUE
SMALL = g.GEMM_F32_ERR_SCRATCH_TOO_SMALL
ACCEPTED = g.GEMM_F32_ERR_NO_DEVICE
COEFFICIENTS = (ctypes.c_float * 192)(*[3.4445, -4.7750, 2.0315] * 64)
INF, NAN = float("inf"), float("nan")
no_device = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not real")


def coefficients(*values):
    return ctypes.addressof((ctypes.c_float * len(values))(*values)), values


BALANCE = dict(dtype=0, tokens=500, groups=48, choices=4, scores=0, sets=6, kept=3, normalize=1, scale=2.5, logits=OK, ld=48,
               bias=None, weights=OK, experts=OK, offsets=OK, order=OK, work=OK, work_bytes=1 << 20, stream=None)
BGRAD = dict(dtype=0, tokens=5, groups=8, choices=2, scores=0, normalize=1, scale=2.5, logits=OK, ld=8, weights=OK, experts=OK,
             grad=OK, dlogits=OK, ldd=8, stream=None)
QUANT = dict(dtype=0, rows=8, k=32, X=OK, layout=0, ld=32, codes=OK, scales=OK, stream=None)
DEQUANT = dict(dtype=0, rows=8, k=32, codes=OK, scales=OK, X=OK, ld=32, stream=None)
LINEAR = dict(dtype=0, m=80, n=16, k=32, groups=2, X=OK, ldx=32, codes=OK, scales=OK, offsets=OK, bias=None, act=0, Y=OK, ldy=16,
              work=OK, work_bytes=1 << 20, stream=None)
ORTHO = dict(dtype=0, batch=2, rows=180, cols=200, X=OK, ldx=200, stride_x=36000, steps=5, f=ctypes.addressof(COEFFICIENTS),
             scale=1.0, Y=OK, ldy=200, stride_y=36000, work=OK, work_bytes=1 << 31, stream=None)

REFUSALS = [
    ("expert_route_balanced", BALANCE, [
        dict(dtype=2), dict(tokens=-1), dict(groups=0), dict(groups=1026, ld=2000), dict(choices=0), dict(choices=25),
        dict(choices=33, groups=96, ld=96), dict(ld=47), dict(scores=2), dict(scores=-1), dict(sets=0), dict(sets=5), dict(sets=96),
        dict(groups=1024, ld=1024, sets=128), dict(kept=0), dict(kept=7), dict(normalize=2), dict(scale=0.0), dict(scale=-1.0),
        dict(scale=INF), dict(scale=NAN), dict(logits=None), dict(logits=OK + 2), dict(bias=OK + 2), dict(weights=None),
        dict(experts=None), dict(offsets=None), dict(order=None), dict(work=None), dict(tokens=1 << 30)]),
    ("expert_route_balanced_grad", BGRAD, [
        dict(dtype=2), dict(tokens=-1), dict(choices=0), dict(choices=9), dict(ld=7), dict(ldd=7), dict(scores=2),
        dict(normalize=-1), dict(scale=0.0), dict(scale=NAN), dict(logits=None), dict(weights=None), dict(experts=None),
        dict(grad=None), dict(dlogits=None)]),
    ("expert_int8_quantize", QUANT, [
        dict(dtype=2), dict(rows=-1), dict(k=0), dict(ld=31), dict(layout=2), dict(layout=1, ld=7), dict(X=None), dict(X=OK + 2),
        dict(codes=None), dict(codes=OK + 4), dict(scales=None), dict(scales=OK + 2)]),
    ("expert_int8_dequantize", DEQUANT, [
        dict(dtype=2), dict(rows=-1), dict(k=0), dict(ld=31), dict(X=None), dict(codes=None), dict(codes=OK + 4),
        dict(scales=None), dict(scales=OK + 1)]),
    ("expert_int8_linear", LINEAR, [
        dict(dtype=2), dict(m=-1), dict(n=0), dict(k=0), dict(k=131073, ldx=131073), dict(groups=0), dict(offsets=None),
        dict(offsets=OK + 2), dict(ldx=31), dict(ldy=15), dict(act=3), dict(act=-1), dict(codes=None), dict(codes=OK + 4),
        dict(scales=None), dict(X=None), dict(Y=None), dict(work=None), dict(work=OK + 4), dict(bias=OK + 2), dict(ldx=1 << 21),
        dict(m=1 << 29, groups=1000)]),
    ("expert_orthogonalize", ORTHO, [
        dict(dtype=2), dict(batch=-1), dict(rows=0), dict(cols=0), dict(ldx=199), dict(ldy=199), dict(stride_x=-1),
        dict(stride_y=35999), dict(steps=0), dict(steps=65), dict(f=None), dict(scale=INF), dict(scale=NAN), dict(X=None),
        dict(Y=None), dict(X=OK + 2), dict(work=None), dict(work=OK + 8), dict(cols=1 << 22, ldx=1 << 22, ldy=1 << 22),
        dict(ldx=1 << 21)]),
]


@pytest.mark.parametrize("name,base,change", [(n, b, c) for n, b, cs in REFUSALS for c in cs])
def test_refuses(name, base, change):
    assert x._functions()[name](*{**base, **change}.values()) == BAD


@pytest.mark.parametrize("name,base", [(n, b) for n, b, _ in REFUSALS])
@no_device
def test_good_arguments_reach_the_device_check(name, base):
    assert x._functions()[name](*base.values()) == ACCEPTED


def test_workspaces():
    f = x._functions()
    space = f["expert_route_balanced_workspace"]
    assert space(128, 512) == 0 and space(0, 8) == 0
    assert space(128, 513) == 4 * 513 * 4                  # parts of 32 tokens, up to 8192 of them
    assert space(129, 8) == 5 * 8 * 4
    assert space(8193, 8) == 65 * 8 * 4                    # then of 128
    assert f["expert_route_balanced"](*{**BALANCE, "work_bytes": 16 * 48 * 4 - 1}.values()) == SMALL
    assert f["expert_int8_workspace"](80, 130) == 80 * (256 + 4) and f["expert_int8_workspace"](0, 130) == 0
    assert f["expert_int8_linear"](*{**LINEAR, "work_bytes": 80 * 132 - 1}.values()) == SMALL
    space = f["expert_orthogonalize_workspace"]
    assert space(0, 5, 64, 256) == 0 and space(1, 5, 100, 128) == 0       # one strip of columns: none
    assert space(0, 5, 300, 60) > 0 and space(0, 0, 300, 300) == 0 and space(3, 1, 300, 300) == 0
    need = space(0, 2, 180, 200)
    assert f["expert_orthogonalize"](*{**ORTHO, "work_bytes": need - 1}.values()) == SMALL
    # A stack's matrices are worked on as many at a time as 2 GiB hold.
    assert space(1, 1000, 2048, 4096) < (5 << 29) and space(1, 1000, 2048, 4096) == space(1, 2000, 2048, 4096)


@no_device
@pytest.mark.parametrize("f,steps,accepted", [
    ((3.4445, -4.7750, 2.0315), 5, True), ((1.5, -0.5, 0.0), 30, True), ((1.875, -1.25, 0.375), 64, True),
    ((30.9, 0.0, 0.0), 1, True), ((31.1, 0.0, 0.0), 1, False), ((5.0, 0.0, 0.0), 2, True), ((8.0, 0.0, 0.0), 2, False),
    ((0.0, 0.0, 30.0), 1, True), ((0.0, 0.0, 32.0), 1, False), ((0.0, -32.0, 0.0), 1, False), ((2.0, 60.0, -60.0), 1, True),
    ((2.0, 130.0, -130.0), 1, False), ((NAN, 0.0, 0.0), 1, False), ((1.0, INF, 0.0), 1, False), ((1.0, 0.0, -INF), 1, False)])
def test_coefficients_that_would_leave_the_range_of_a_plane(f, steps, accepted):
    """Entries of X, A and a I + b A + c A A stay below 31: 8 s takes 1 to 8, whose square is 64;
    2 + 60 u - 60 u^2 is 17 at its turn, 2 + 130 u - 130 u^2 is 34.5."""
    address, keep = coefficients(*(f * steps))
    array = (ctypes.c_float * (3 * steps))(*(f * steps))
    status = x._functions()["expert_orthogonalize"](*{**ORTHO, "steps": steps, "f": ctypes.addressof(array)}.values())
    assert status == (ACCEPTED if accepted else BAD)


def test_what_the_binding_refuses():
    a = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        g.route_balanced(a, 2)
    with pytest.raises(ValueError):
        g.int8_quantize(a)
    with pytest.raises(ValueError):
        g.orthogonalize(a)
    with pytest.raises(TypeError):
        g.route_balanced(a.half(), 2)
    with pytest.raises(TypeError):
        g.int8_quantize(a.double())
    with pytest.raises(TypeError):
        g.orthogonalize(a.int())
    with pytest.raises(TypeError):
        g.orthogonalize([[1.0]])
    with pytest.raises(KeyError):
        g.route_balanced(a, 2, scores="tanh")
    with pytest.raises(TypeError):
        g.int8_dequantize(g.Int8Tensor(torch.zeros((4, 16), dtype=torch.int8), torch.zeros(4), 10), dtype=torch.half)
    with pytest.raises(KeyError):
        g.int8_linear(a, g.Int8Tensor(torch.zeros((4, 16), dtype=torch.int8), torch.zeros(4), 8), activation="tanh")


@pytest.mark.parametrize("codes,scales,k", [
    ((4, 16), (4,), 17), ((4, 32), (4,), 16), ((4, 16), (5,), 10), ((4, 16), (4, 1), 10), ((2, 4, 16), (2, 5), 10),
    ((2, 4, 16), (8,), 10), ((4, 16), (4,), 0), ((16,), (), 16)])
def test_int8_tensor_shapes(codes, scales, k):
    with pytest.raises(ValueError):
        g.Int8Tensor(torch.zeros(codes, dtype=torch.int8), torch.zeros(scales), k)


def test_int8_tensor():
    q = g.Int8Tensor(torch.zeros((3, 5, 208), dtype=torch.int8), torch.zeros((3, 5)), 200)
    assert tuple(q.shape) == (3, 5, 200)
    with pytest.raises(TypeError):
        g.Int8Tensor(torch.zeros((5, 16), dtype=torch.uint8), torch.zeros(5), 10)
    with pytest.raises(TypeError):
        g.Int8Tensor(torch.zeros((5, 16), dtype=torch.int8), torch.zeros(5).double(), 10)
    with pytest.raises(ValueError):
        g.Int8Tensor(torch.zeros((16, 5), dtype=torch.int8).t(), torch.zeros(5), 10)


@no_device
def test_largest_calls():
    """What the kernels count in 32 bits fits, or the call is refused."""
    f = x._functions()
    most = {**BALANCE, "groups": 32, "ld": 32, "sets": 1, "kept": 1, "choices": 32, "work_bytes": 1 << 40}
    assert f["expert_route_balanced"](*{**most, "tokens": 67108801}.values()) == BAD
    assert f["expert_route_balanced"](*{**most, "tokens": (2 ** 31 - 2048) // 32}.values()) == ACCEPTED
    args = {**LINEAR, "work_bytes": 1 << 50}
    assert f["expert_int8_linear"](*{**args, "m": 700000, "groups": 60000}.values()) == BAD
    assert f["expert_int8_linear"](*{**args, "m": 700000, "groups": 44000}.values()) == ACCEPTED
    args = {**ORTHO, "work_bytes": 1 << 62, "ldx": 1 << 20, "ldy": 1 << 20, "batch": 1}
    assert f["expert_orthogonalize"](*{**args, "rows": 1 << 17, "cols": 1 << 18}.values()) == ACCEPTED
    assert f["expert_orthogonalize"](*{**args, "rows": 1 << 18, "cols": 1 << 18}.values()) == BAD
    assert f["expert_orthogonalize"](*{**args, "rows": 64, "cols": 1 << 20}.values()) == ACCEPTED
