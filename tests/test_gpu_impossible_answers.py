"""Answers of probability 0 in the preference loss (needs an MI355X): a token
whose logit is -inf makes its sequence's log probability -inf and z infinite."""
from __future__ import annotations

import math

import pytest
import torch

from gpu_helpers import DEV, require_gpu
from kronecker_sparse_structured_amd import libks

pytestmark = pytest.mark.gpu
INF = float("inf")


def losses(impossible, smoothing, dtype=torch.float32):
    """One pair of two-token answers over 8 equal logits; `impossible`: the
    sequence (0 chosen, 1 rejected) that has a token of probability 0."""
    x = torch.zeros(2, 2, 8, dtype=dtype, device=DEV)
    labels = torch.ones(2, 2, dtype=torch.int64, device=DEV)
    if impossible is not None:
        x[impossible, 1, 1] = -INF
    return libks.preference_loss(x, labels, torch.zeros(2, 2, device=DEV), beta=0.5, smoothing=smoothing)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("impossible,smoothing,want", [
    (1, 0.0, 0.0), (0, 0.0, INF), (1, 1.0, INF), (0, 1.0, 0.0), (1, 0.25, INF), (0, 0.25, INF)])
def test_loss_is_the_limit(impossible, smoothing, want, dtype):
    require_gpu()
    loss, rewards, tokens, d = losses(impossible, smoothing, dtype)
    assert float(loss) == want
    assert float(rewards[impossible]) == -INF and math.isfinite(float(rewards[1 - impossible]))
    # the slope of each side is 0 or its weight: finite, and 0 where the loss is settled
    assert torch.isfinite(d).all() and (want != 0.0 or not d.any())


def test_both_answers_impossible_are_not_a_number():
    require_gpu()
    x = torch.zeros(2, 2, 8, device=DEV)
    x[:, 1, 1] = -INF
    labels = torch.ones(2, 2, dtype=torch.int64, device=DEV)
    assert torch.isnan(libks.preference_loss(x, labels, torch.zeros(2, 2, device=DEV))[0])
