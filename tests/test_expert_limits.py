"""Largest calls that the expert-layer entry points accept: what their kernels
count in 32 bits has to fit, or the call is refused before anything is
launched (no GPU compute: without a device an accepted call ends at the device
check)."""
import pytest
import torch

import dense_gemm_optimisation_fp32_amd as g
from dense_gemm_optimisation_fp32_amd import expert_ops as x

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not real")

OK = 0x10000            # a well aligned address that is never followed
BAD = g.GEMM_F32_ERR_INVALID_VALUE
ACCEPTED = g.GEMM_F32_ERR_NO_DEVICE


def route(tokens, groups, choices):
    return x._functions()["expert_route"](0, tokens, groups, choices, 1, OK, groups, OK, OK, OK, OK, OK, 1 << 40, None)


def route_grad(tokens, groups, choices):
    return x._functions()["expert_route_grad"](0, tokens, groups, choices, 1, OK, groups, OK, OK, OK, OK, groups, None)


@pytest.mark.parametrize("tokens,choices", [(67108863, 32), (67108801, 32), (134217721, 16)])
def test_slot_counters_of_a_workgroup_stay_in_32_bits(tokens, choices):
    """A workgroup of 1024 threads steps its slot counters past the last slot:
    up to 2^31 - 2048 slots they do not wrap."""
    assert tokens * choices > 2 ** 31 - 2048
    assert route(tokens, 32, choices) == BAD
    assert route((2 ** 31 - 2048) // choices, 32, choices) == ACCEPTED


def weight_grad(groups, k=32, n=16):
    return x._functions()["expert_grouped_weight_grad"](0, 8, n, k, groups, OK, k, OK, n, OK, OK, n, k * n, None)


@pytest.mark.parametrize("groups", [1 << 30, 1 << 29, 600_000_000, (1 << 28) + 1])
def test_weight_gradient_workgroups_are_counted_in_32_bits(groups):
    """Every XCD takes a share of every expert's tiles: at least eight
    workgroups an expert, also where it has one tile."""
    assert weight_grad(groups) == BAD
    assert weight_grad(1 << 16) == ACCEPTED
