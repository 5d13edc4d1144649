"""In-place use of what the differentiable preference loss returns (needs an
MI355X): gradient accumulation divides the loss, logging rescales the rewards."""
from __future__ import annotations

import pytest
import torch

from gpu_helpers import DEV, require_gpu
from kronecker_sparse_structured_amd import layer, libks

pytestmark = pytest.mark.gpu


def problem():
    g = torch.Generator().manual_seed(4)
    logits = torch.randn(4, 6, 50, generator=g).to(DEV)
    labels = torch.randint(50, (4, 6), generator=g).to(DEV)
    return logits, labels, (-4 * torch.rand(4, 6, generator=g)).to(DEV)


def gradient(change):
    logits, labels, ref = problem()
    logits.requires_grad_(True)
    results = list(layer.preference_loss(logits, labels, ref))
    change(results)
    results[0].backward()
    return logits.grad, results


def halve(r):
    r[0] /= 2


def add(r):
    r[0] += r[0].detach()


def rescale(r):
    r[1].div_(0.1)
    r[2].mul_(3).zero_()


@pytest.mark.parametrize("change,factor", [(halve, 0.5), (add, 1.0), (rescale, 1.0)])
def test_results_may_be_changed_before_backward(change, factor):
    require_gpu()
    want, was = gradient(lambda r: None)
    got, now = gradient(change)
    assert torch.equal(got, want * factor) and want.any()     # a power of two: exact
    if change is not rescale:
        assert torch.equal(was[1], now[1]) and torch.equal(was[2], now[2])


def test_results_have_memory_of_their_own():
    require_gpu()
    logits, labels, ref = problem()
    for results in (layer.preference_loss(logits, labels, ref), libks.preference_loss(logits, labels, ref)):
        at = [t.untyped_storage().data_ptr() for t in results]
        assert len(set(at)) == len(at) and not any(t._is_view() for t in results)
        versions = [t._version for t in results]
        results[1].mul_(2)
        versions[1] += 1
        assert [t._version for t in results] == versions
