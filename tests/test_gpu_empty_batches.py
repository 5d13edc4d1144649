"""Batches without rows (needs an MI355X): gradients of the weights are zeros,
with whatever handle, and a workspace of no bytes need not exist."""
from __future__ import annotations

import ctypes

import pytest
import torch

from gpu_helpers import DEV, require_gpu
from kronecker_sparse_structured_amd import layer, libks
from test_gpu_adapters import BF16, F32, PAIR, draw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("patterns", [PAIR, [(3, 5, 7, 2)]], ids=["pair", "factor"])
@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("transposed", [False, True])
def test_a_chain_without_rows(patterns, t, transposed):
    require_gpu()
    n_in, n_out = patterns[0][0] * patterns[0][2] * patterns[0][3], patterns[-1][0] * patterns[-1][1] * patterns[-1][3]
    X, A, B, scale, ids = draw(0, n_in, n_out, 3, 5, t, t)
    Ws = [torch.randn(a, d, b, c).to(t).to(DEV) for a, b, c, d in patterns]
    chain = libks.AdapterChain(Ws, patterns, A, B, scale, transposed=transposed)
    Y, H = chain.matmul(X, ids, keep=True)
    dY = torch.empty(0, n_out, device=DEV)
    for _ in range(2):
        junk = [torch.full(t.shape, 7.0, device=DEV) for t in (A, B)]     # the outputs' memory is not zero before
        del junk
        dX, dA, dB = chain.backward(dY, X, H, ids)
        assert dX.shape == X.shape and not dA.any() and not dB.any()
    assert chain.backward(dY, X, H, ids, weights=False)[1:] == (None, None)


def test_a_layer_without_rows():
    require_gpu()
    m = layer.AdapterLinear(layer.KSLinear([(3, 5, 7, 2)], device=DEV), 3, 5)
    x = torch.empty(2, 0, 42, device=DEV, requires_grad=True)
    y = m(x, torch.empty(2, 0, dtype=torch.int32, device=DEV))
    assert y.shape == (2, 0, 30)
    y.sum().backward()
    assert x.grad.shape == x.shape and not m.A.grad.any() and not m.B.grad.any()


def test_no_workspace_where_none_is_needed():
    require_gpu()
    _, A, B, scale, _ = draw(0, 42, 30, 3, 5, F32, F32)
    ad = libks._adapters(A, B, scale, 42, 30)
    lib, size = libks.load(), ctypes.c_size_t(1)
    assert lib.ks_adapter_backward_workspace_size(ad, 0, size) == libks.KS_OK and size.value == 0
    dA, dB = torch.full(A.shape, 7.0, device=DEV), torch.full(B.shape, 7.0, device=DEV)
    assert lib.ks_adapter_backward(ad, None, None, None, None, None, dA.data_ptr(), dB.data_ptr(), 0, libks.DTYPE_F32, None,
                                   0, libks._raw_stream(0)) == libks.KS_OK
    assert not dA.any() and not dB.any()
