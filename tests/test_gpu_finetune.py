"""Adapters, preference loss and AdamW together (needs an MI355X): the example
learns its tasks, with either width of the moments."""
import pytest

from gpu_helpers import require_gpu
from kronecker_sparse_structured_amd import finetune

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [8, 32])
def test_the_example_learns(bits):
    require_gpu()
    out = finetune.run(steps=40, state_bits=bits)
    # no adapter has learned anything at first: the policy is the reference
    assert abs(out["loss"][0] - 0.6931) < 1e-3 and abs(out["margin"][0]) < 1e-2
    assert sum(out["loss"][-5:]) / 5 < 0.35 and out["margin"][-1] > 1.0
    again = finetune.run(steps=5, state_bits=bits)
    assert again["loss"] == out["loss"][:5]        # the same steps give the same bits
