"""Gradients through libks are formed outside autograd (needs an MI355X): asking
for a derivative of one raises, where it would come out as zero."""
from __future__ import annotations

import pytest
import torch

from gpu_helpers import DEV, require_gpu
from kronecker_sparse_structured_amd import layer

pytestmark = pytest.mark.gpu


def ks_layer(x):
    return layer.KSLinear([(3, 5, 7, 2)], device=DEV)(x).square().sum()


def adapters(x):
    m = layer.AdapterLinear(layer.KSLinear([(3, 5, 7, 2)], device=DEV), 2, 3)
    return m(x, torch.zeros(8, dtype=torch.int32, device=DEV)).square().sum()


def preference(x):
    labels = torch.zeros(2, 4, dtype=torch.int64, device=DEV)
    return layer.preference_loss(x.view(2, 4, 42), labels, torch.zeros(2, 4, device=DEV))[0]


@pytest.mark.parametrize("f", [ks_layer, adapters, preference])
def test_second_derivative_raises(f):
    require_gpu()
    x = torch.randn(8, 42, device=DEV, requires_grad=True)
    first, = torch.autograd.grad(f(x), x, create_graph=True)
    assert first.any()
    with pytest.raises(RuntimeError, match="only first derivatives"):
        first.square().sum().backward()
    value = f(x)
    first, = torch.autograd.grad(value, x, create_graph=True)
    with pytest.raises(RuntimeError, match="only first derivatives"):
        (value + 0.1 * first.norm()).backward()              # a gradient penalty
    # the first alone is as it was
    again, = torch.autograd.grad(f(x), x)
    assert torch.isfinite(again).all()


def test_first_derivatives_with_a_graph_are_those_without():
    require_gpu()
    m = layer.KSLinear([(3, 5, 7, 2), (1, 4, 30, 1)], device=DEV)
    x = torch.randn(8, 42, device=DEV, requires_grad=True)
    args = (x, *m.weights)
    want = torch.autograd.grad(m(x).square().sum(), args)
    got = torch.autograd.grad(m(x).square().sum(), args, create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
