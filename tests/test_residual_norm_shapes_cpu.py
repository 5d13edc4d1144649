"""Shapes that layer.ResidualNorm takes and refuses, on the CPU: the module's own
code over a stand-in for the handle that computes in torch and has the handle's
checks."""
from __future__ import annotations

import pytest
import torch

from kronecker_sparse_structured_amd import layer, libks


class Handle:
    """z = x + residual gate y and h = z (the norms are left out), over rows."""

    def __init__(self, width, *vectors, kind, eps, residual):
        self.width, self.residual = width, residual

    def forward(self, x, y=None, gate=None, dtype=None, keep=False):
        assert x.dim() == 2 and x.shape[1] == self.width
        if y is None:
            if gate is not None:
                raise ValueError("a gate needs a y")
            return x, x.clone()
        assert y.shape == x.shape
        rows = len(x)
        u = y
        if gate is not None:
            assert gate.dim() == 2 and gate.shape[1] == self.width
            groups = gate.shape[0]
            assert (groups > 0 or rows == 0) and (groups == 0 or rows % groups == 0)
            u = u * gate.repeat_interleave(rows // groups if groups else 0, 0)
        z = x + self.residual * u
        return z, z.clone()


@pytest.fixture
def norm(monkeypatch):
    monkeypatch.setattr(libks, "ResidualNorm", Handle)
    return layer.ResidualNorm(8, params=torch.float32).requires_grad_(False)


# what the gate's or the block's values would be read from as rows of 8, one after another
GATES = [(4, 16), (24,), (2, 4), (4, 6, 4), (4, 1, 16), (48, 4), (4, 6, 1, 8), (4, 6, 8, 1), (1, 4, 6, 8), (6, 8), (1, 6, 8), (4, 3, 8), ()]


@pytest.mark.parametrize("gate", GATES, ids=str)
def test_a_gate_of_another_shape_is_refused(norm, gate):
    x = torch.randn(4, 6, 8)
    with pytest.raises(ValueError):
        norm(x, torch.randn(4, 6, 8), torch.randn(gate))


@pytest.mark.parametrize("y", [(6, 4, 8), (4, 3, 16), (4, 6, 4), (24, 8), (192,), (4, 1, 8), (8,), (4, 6, 8, 1)], ids=str)
def test_a_block_of_another_shape_is_refused(norm, y):
    with pytest.raises(ValueError):
        norm(torch.randn(4, 6, 8), torch.randn(y))


@pytest.mark.parametrize("x", [(4, 6, 16), (4, 6, 4), (24, 1), (16,), (0, 16), ()], ids=str)
def test_rows_of_another_width_are_refused(norm, x):
    x = torch.randn(x)
    with pytest.raises(ValueError):
        norm(x)
    with pytest.raises(ValueError):
        norm(x, x.clone())
    with pytest.raises(ValueError):
        layer.ResidualNorm(8, pre=False)(x)          # with nothing to compute too


@pytest.mark.parametrize("gate", [(4, 6, 8), (4, 8), (4, 1, 8), (1, 8), (1, 1, 8), (8,)], ids=str)
def test_the_shapes_that_are_meant(norm, gate):
    x, y, g = torch.randn(4, 6, 8), torch.randn(4, 6, 8), torch.randn(gate)
    z, h = norm(x, y, g)
    wide = g if gate != (4, 8) else g[:, None, :]
    assert torch.equal(z, x + y * wide) and h.shape == x.shape
    z, h = norm(x.transpose(0, 1), y.transpose(0, 1))
    assert torch.equal(z, (x + y).transpose(0, 1)) and h.shape == (6, 4, 8)


def test_one_row_and_none(norm):
    x, y = torch.randn(8), torch.randn(8)
    assert torch.equal(norm(x, y, torch.ones(8))[0], x + y)
    for shape, gate in (((0, 8), (0, 8)), ((0, 5, 8), (0, 8)), ((4, 0, 8), (4, 8)), ((4, 0, 8), (8,))):
        z, h = norm(torch.ones(shape), torch.ones(shape), torch.ones(gate))
        assert z.shape == shape and h.shape == shape


def test_a_gate_without_a_block_is_refused(norm):
    x = torch.randn(4, 6, 8)
    for m in (norm, layer.ResidualNorm(8, pre=False)):       # with nothing to compute too
        with pytest.raises(ValueError):
            m(x, gate=torch.ones(4, 8))
