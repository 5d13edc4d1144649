"""Forward-mode derivatives through the layers, on the CPU over stand-ins for the
library's calls: none is formed, so a tangent raises where it would be dropped and
its derivative read as zero; without a tangent the layers run inside a dual level."""
from __future__ import annotations

import pytest
import torch
from torch.autograd import forward_ad

from kronecker_sparse_structured_amd import layer, libks

PATTERNS = [(1, 4, 2, 4), (4, 2, 4, 1)]      # 8 -> 16 -> 8


@pytest.fixture(autouse=True)
def library(monkeypatch):
    class Norm:
        def __init__(self, width, *vectors, **options):
            pass

        def forward(self, x, y=None, gate=None, dtype=None, keep=False):
            return x.detach().clone(), x.detach().clone()

    class Chain:
        def __init__(self, *args, **options):
            pass

        def matmul(self, X, ids):
            return torch.zeros(len(X), 8)

    monkeypatch.setattr(libks, "ResidualNorm", Norm)
    monkeypatch.setattr(libks, "AdapterChain", Chain)
    monkeypatch.setattr(libks, "matmul", lambda X, W, p: torch.zeros(len(X), p[0] * p[1] * p[3]))
    monkeypatch.setattr(libks, "chain_matmul", lambda X, Ws, ps: torch.zeros(len(X), 8))


def linear():
    return layer.KSLinear(PATTERNS).requires_grad_(False)


def adapters():
    return layer.AdapterLinear(linear(), 3, 2).requires_grad_(False)


def call(m, x, y=None, gate=None):
    if isinstance(m, layer.AdapterLinear):
        return m(x, torch.zeros(x.shape[:-1], dtype=torch.int32))
    return m(x) if isinstance(m, layer.KSLinear) else m(x, y, gate)


def norm():
    return layer.ResidualNorm(8, post=True, scale=0.5).requires_grad_(False)


@pytest.mark.parametrize("make", [linear, adapters, norm])
@pytest.mark.parametrize("grad", [True, False], ids=["grad", "no_grad"])
def test_a_tangent_of_the_input_raises(make, grad):
    m, x = make(), torch.randn(5, 8)
    with forward_ad.dual_level(), torch.set_grad_enabled(grad):
        call(m, x, x, torch.ones(5, 8))
        with pytest.raises(NotImplementedError):
            call(m, forward_ad.make_dual(x, torch.ones_like(x)), x)
    call(m, x, x)


@pytest.mark.parametrize("make", [linear, adapters, norm])
def test_a_tangent_of_a_parameter_raises(make):
    m, x = make(), torch.randn(5, 8)
    for name, p in m.named_parameters():
        with forward_ad.dual_level():
            dual = forward_ad.make_dual(p.detach(), torch.ones_like(p))
            with pytest.raises(NotImplementedError):
                torch.func.functional_call(m, {name: dual}, (x, torch.zeros(5, dtype=torch.int32))
                                           if make is adapters else (x,) if make is linear else (x, x))


def test_a_tangent_of_the_block_or_its_gate_raises():
    x = torch.randn(5, 8)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        for y, gate in ((dual, None), (x, dual)):
            with pytest.raises(NotImplementedError):
                norm()(x, y, gate)
            with pytest.raises(NotImplementedError):
                layer.ResidualNorm(8, pre=False)(x, y, gate)
    plain = layer.ResidualNorm(8, pre=False)
    with forward_ad.dual_level():                    # x itself, tangent and all: nothing is computed
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        assert forward_ad.unpack_dual(plain(dual)[0]).tangent is not None


def test_a_tangent_of_the_gradient_raises(monkeypatch):
    """The derivative of a backward pass by what it is given."""
    monkeypatch.setattr(libks, "matmul_dx", lambda dY, W, p: torch.zeros(len(dY), 8))
    x = torch.randn(5, 8, requires_grad=True)
    y = layer.ks_matmul_autograd(x, torch.randn(1, 4, 4, 2), PATTERNS[0])
    torch.autograd.grad(y, x, torch.ones_like(y), retain_graph=True)
    with forward_ad.dual_level():
        upstream = forward_ad.make_dual(torch.ones_like(y), torch.ones_like(y))
        for create_graph in (False, True):
            with pytest.raises(NotImplementedError):
                torch.autograd.grad(y, x, upstream, retain_graph=True, create_graph=create_graph)
