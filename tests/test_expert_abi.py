"""Host-side checks of the expert-layer operators (no GPU compute): the header
and the binding agree, and every entry point refuses bad arguments before it
touches a device or an operand."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import dense_gemm_optimisation_fp32_amd as g
from dense_gemm_optimisation_fp32_amd import expert_ops as x

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "expert_ops.h")
OK = 0x10000            # a well aligned address that is never followed
BAD = g.GEMM_F32_ERR_INVALID_VALUE
SMALL = g.GEMM_F32_ERR_SCRATCH_TOO_SMALL


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(expert_[a-z0-9_]+)\s*\(", text)))


def test_header_binding_and_library_agree():
    assert declared() == sorted(g.EXPERT_FUNCTIONS)
    lib = ctypes.CDLL(g.LIB_PATH)
    for name in declared():
        assert hasattr(lib, name), f"{name} not exported"


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "expert_ops.h"\nint main(void){return EXPERT_BF16 - 1 + GEMM_F32_SUCCESS;}\n')
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.dirname(HEADER), "-c", str(src), "-o",
                        str(tmp_path / "t.o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


# Arguments of each call that would be accepted, by position.
LINEAR = dict(dtype=0, m=8, n=16, k=32, groups=2, A=OK, lda=32, B=OK, layout=0, ldb=16, stride=512, offsets=OK,
              bias=None, act=0, C=OK, ldc=16, stream=None)
WGRAD = dict(dtype=0, m=8, n=16, k=32, groups=2, A=OK, lda=32, G=OK, ldg=16, offsets=OK, dB=OK, ldd=16, stride=512,
             stream=None)
QUANT = dict(dtype=0, rows=8, k=32, X=OK, layout=0, ld=32, codes=OK, scales=OK, stream=None)
DEQUANT = dict(dtype=0, rows=8, k=32, codes=OK, scales=OK, X=OK, ld=32, stream=None)
MX4 = dict(dtype=0, m=80, n=16, k=32, groups=2, X=OK, ldx=32, codes=OK, scales=OK, offsets=OK, bias=None, act=0,
           Y=OK, ldy=16, work=OK, work_bytes=1 << 20, stream=None)
ROUTE = dict(dtype=0, tokens=500, groups=8, choices=2, normalize=1, logits=OK, ld=8, weights=OK, experts=OK,
             offsets=OK, order=OK, work=OK, work_bytes=1 << 20, stream=None)
RGRAD = dict(dtype=0, tokens=5, groups=8, choices=2, normalize=1, logits=OK, ld=8, weights=OK, experts=OK, grad=OK,
             dlogits=OK, ldd=8, stream=None)

REFUSALS = [
    ("expert_grouped_linear", LINEAR, [
        dict(dtype=2), dict(dtype=-1), dict(m=-1), dict(n=0), dict(k=0), dict(groups=0), dict(lda=31), dict(ldb=15),
        dict(layout=1, ldb=31), dict(layout=2), dict(ldc=15), dict(stride=-1), dict(offsets=None), dict(offsets=OK + 2),
        dict(A=None), dict(B=None), dict(C=None), dict(A=OK + 2), dict(dtype=1, A=OK + 1), dict(bias=OK + 1),
        dict(act=3), dict(act=-1), dict(m=1 << 31), dict(lda=1 << 21), dict(k=1 << 15, n=1 << 15, lda=1 << 15,
                                                                            ldb=1 << 15, ldc=1 << 15)]),
    ("expert_grouped_weight_grad", WGRAD, [
        dict(dtype=3), dict(m=-1), dict(n=0), dict(k=0), dict(groups=0), dict(lda=31), dict(ldg=15), dict(ldd=15),
        dict(offsets=None), dict(A=None), dict(G=None), dict(dB=None), dict(dB=OK + 2), dict(ldg=1 << 21),
        dict(k=1 << 15, n=1 << 15, lda=1 << 15, ldg=1 << 15, ldd=1 << 15)]),
    ("expert_mx4_quantize", QUANT, [
        dict(dtype=2), dict(rows=-1), dict(k=0), dict(ld=31), dict(layout=2), dict(layout=1, ld=7), dict(X=None),
        dict(X=OK + 2), dict(codes=None), dict(codes=OK + 4), dict(scales=None), dict(rows=1 << 30, k=1 << 10)]),
    ("expert_mx4_dequantize", DEQUANT, [
        dict(dtype=2), dict(rows=-1), dict(k=0), dict(ld=31), dict(X=None), dict(codes=None), dict(codes=OK + 4),
        dict(scales=None), dict(scales=OK + 1)]),
    ("expert_mx4_linear", MX4, [
        dict(dtype=2), dict(m=-1), dict(n=0), dict(k=0), dict(groups=0), dict(offsets=None), dict(ldx=31),
        dict(ldy=15), dict(act=3), dict(codes=None), dict(codes=OK + 4), dict(scales=None), dict(X=None),
        dict(Y=None), dict(work=None), dict(work=OK + 4), dict(bias=OK + 2), dict(ldx=1 << 21)]),
    ("expert_route", ROUTE, [
        dict(dtype=2), dict(tokens=-1), dict(groups=0), dict(groups=1025, ld=2000), dict(choices=0), dict(choices=9),
        dict(groups=64, ld=64, choices=33), dict(ld=7), dict(normalize=2), dict(logits=None), dict(weights=None),
        dict(experts=None), dict(offsets=None), dict(order=None), dict(work=None), dict(tokens=1 << 30, choices=4)]),
    ("expert_route_grad", RGRAD, [
        dict(dtype=2), dict(tokens=-1), dict(choices=0), dict(choices=9), dict(ld=7), dict(ldd=7), dict(normalize=-1),
        dict(logits=None), dict(weights=None), dict(experts=None), dict(grad=None), dict(dlogits=None)]),
]


@pytest.mark.parametrize("name,base,change", [(n, b, c) for n, b, cs in REFUSALS for c in cs])
def test_refuses(name, base, change):
    assert x._functions()[name](*{**base, **change}.values()) == BAD


@pytest.mark.parametrize("name,base", [(n, b) for n, b, _ in REFUSALS])
@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not real")
def test_good_arguments_reach_the_device_check(name, base):
    assert x._functions()[name](*base.values()) == g.GEMM_F32_ERR_NO_DEVICE


def test_workspaces():
    f = x._functions()
    assert f["expert_mx4_workspace"](80, 16, 32, 2) == 80 * (64 + 4)      # codes and scales of 128 columns
    assert f["expert_mx4_workspace"](32, 16, 32, 2) == 0                  # few rows an expert: no copy of x
    assert f["expert_mx4_workspace"](0, 16, 32, 2) == 0
    assert f["expert_mx4_linear"](*{**MX4, "work_bytes": 80 * 68 - 1}.values()) == SMALL
    assert f["expert_route_workspace"](128, 8) == 0
    assert f["expert_route_workspace"](129, 8) == 2 * 8 * 4
    assert f["expert_route"](*{**ROUTE, "work_bytes": 4 * 8 * 4 - 1}.values()) == SMALL


def test_binding_refuses_cpu_tensors_and_types():
    off = torch.zeros(3, dtype=torch.int32)
    a, b = torch.zeros(4, 8), torch.zeros(2, 8, 6)
    with pytest.raises(ValueError):
        g.grouped_linear(a, b, off)
    with pytest.raises(ValueError):
        g.grouped_weight_grad(a, torch.zeros(4, 6), off)
    with pytest.raises(ValueError):
        g.mx4_quantize(a)
    with pytest.raises(ValueError):
        g.route(a, 2)
    with pytest.raises(TypeError):
        g.grouped_linear(a.double(), b.double(), off)
    with pytest.raises(TypeError):
        g.mx4_quantize(a.half())
    with pytest.raises(TypeError):
        g.route(a.int(), 2)


@pytest.mark.parametrize("codes,scales,k", [
    ((4, 64), (1, 4, 4), 129), ((4, 128), (1, 4, 4), 129), ((4, 64), (1, 5, 4), 100), ((4, 64), (4, 4), 100),
    ((2, 4, 64), (1, 4, 4), 100), ((2, 4, 64), (3, 1, 4, 4), 100), ((4, 64), (1, 4, 4), 0),
])
def test_mx4_tensor_shapes(codes, scales, k):
    with pytest.raises(ValueError):
        g.Mx4Tensor(torch.zeros(codes, dtype=torch.uint8), torch.zeros(scales, dtype=torch.uint8), k)


def test_mx4_tensor():
    q = g.Mx4Tensor(torch.zeros((3, 5, 128), dtype=torch.uint8), torch.zeros((3, 2, 5, 4), dtype=torch.uint8), 200)
    assert tuple(q.shape) == (3, 5, 200)
    with pytest.raises(TypeError):
        g.Mx4Tensor(torch.zeros((5, 64)), torch.zeros((1, 5, 4)), 100)


@pytest.mark.parametrize("name,base,m,groups,ok", [
    (n, b, m, e, ok) for n, b in (("expert_grouped_linear", LINEAR), ("expert_mx4_linear", MX4))
    for m, e, ok in ((1 << 29, 1000, False), (1 << 25, 1000, True), (700000, 60000, False), (700000, 44000, True))])
@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not real")
def test_row_tiles_are_counted_in_32_bits(name, base, m, groups, ok):
    """Unsorted offsets can make every expert seem to own all rows: the sum of
    such row tiles has to fit as well."""
    args = dict(base, m=m, groups=groups)
    if "work" in args:
        args["work_bytes"] = 1 << 40
    status = x._functions()[name](*args.values())
    assert (status == BAD) != ok
