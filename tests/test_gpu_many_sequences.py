"""More sequences than a grid of one wave each can count (needs an MI355X): their
totals are summed in several launches."""
from __future__ import annotations

import pytest
import torch

from gpu_helpers import DEV, require_gpu
from kronecker_sparse_structured_amd import libks

pytestmark = pytest.mark.gpu


def test_totals_of_more_than_2_26_sequences():
    require_gpu()
    S = (1 << 26) + 5
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(S, 1, 2, device=DEV, generator=g, dtype=torch.bfloat16)
    labels = torch.zeros(S, 1, dtype=torch.int64, device=DEV)
    labels[::3] = 1
    total, tokens = libks.sequence_logp(x, labels)
    # one token a sequence: its log probability, to the bit
    assert torch.equal(total, tokens[:, 0])
    for rows in (slice(0, 1000), slice(S - 1000, S), slice((1 << 25) - 500, (1 << 25) + 500)):
        want = torch.log_softmax(x[rows, 0].double(), 1).gather(1, labels[rows])[:, 0]
        # two exponentials, their sum and its logarithm: 16 ulp of values up to 16
        assert float((total[rows].double() - want).abs().max()) <= 16 * 2.0 ** -23 * 16
