"""Values that no fp32 kernel can take, refused on the host before any HIP call."""
import pytest

import test_stack_abi_cpu as abi
from kronecker_sparse_structured_amd import libks


@pytest.mark.parametrize("residual", [3.5e38, -3.5e38, 1e300, float("inf"), float("-inf")])
def test_a_residual_factor_past_fp32_is_refused(residual):
    """As fp32 it is infinite, and infinity times a value of 0 is NaN."""
    assert abi.forward(abi.norm_struct(residual=residual)) == libks.KS_ERR_INVALID
    assert abi.backward(abi.norm_struct(residual=residual)) == libks.KS_ERR_INVALID
