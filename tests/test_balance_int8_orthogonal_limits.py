"""Limits of 8-bit quantisation and orthogonalising that go by what the kernels count in
32 bits or hold in half precision (no GPU compute): beyond them a call is refused before
it touches a device, within them it reaches the device check."""
import pytest
import torch

import dense_gemm_optimisation_fp32_amd as g
from dense_gemm_optimisation_fp32_amd import expert_ops as x

OK = 0x10000            # a well aligned address that is never followed
BAD = g.GEMM_F32_ERR_INVALID_VALUE
ACCEPTED = g.GEMM_F32_ERR_NO_DEVICE
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not real")


def wraps(k, step):
    """Whether columns counted in `step` pass 2^31 - 1 before the loop over them ends."""
    padded = (k + 15) // 16 * 16
    return (padded + step - 1) // step * step > 2 ** 31 - 1


@pytest.mark.parametrize("k,accepted", [(2 ** 31 - 2049, True), (2 ** 31 - 2047, False), (2 ** 31 - 1500, False), (2 ** 31 - 1, False)])
@pytest.mark.parametrize("layout", [0, 1])
def test_columns_of_a_quantised_matrix(k, accepted, layout):
    """Rows are taken in pieces of 2048 columns."""
    assert accepted or wraps(k, 2048)
    assert not accepted or not wraps(k, 2048)
    status = x._functions()["expert_int8_quantize"](0, 2, k, OK, layout, 2 if layout else k, OK, OK, None)
    assert status == (ACCEPTED if accepted else BAD)
