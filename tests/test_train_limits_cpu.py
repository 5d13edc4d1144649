"""Limits of the adapters' gradients, without a GPU: what no grid can hold is
refused by the size query, and by the call before anything is launched."""
import ctypes

import pytest

from kronecker_sparse_structured_amd import libks

P = dict(A=1 << 40, B=2 << 40, scale=3 << 40, ids=4 << 40, dY=5 << 40, X=6 << 40, H=7 << 40, dX=8 << 40, dA=9 << 40,
         dB=10 << 40, ws=11 << 40, W=12 << 40)


def adapters(n_in, n_out, count=65535, rank=1):
    return libks.ks_adapters_t(P["A"], P["B"], P["scale"], n_in, n_out, rank, count)


def sizes(n_in, n_out, batch):
    """Status of both size queries, and the bytes of the first."""
    lib, a, b = libks.load(), ctypes.c_size_t(0), ctypes.c_size_t(0)
    ad = adapters(n_in, n_out)
    pats = libks._patterns([(1, n_out, n_in, 1)])
    return (lib.ks_adapter_backward_workspace_size(ad, batch, a),
            lib.ks_chain_adapter_backward_workspace_size(pats, 1, ad, batch, libks.DTYPE_F32, 0, b), a.value)


@pytest.mark.parametrize("n_in,n_out", [(16448, 4), (4, 16448)])
def test_refused_before_anything_is_launched(n_in, n_out):
    lib = libks.load()
    # 64-value column groups x (65535 adapters + a slot a block of rows): 255 fit, 257 do not
    assert sizes(16320 if n_in > 4 else 4, 16320 if n_out > 4 else 4, 100)[:2] == (libks.KS_OK, libks.KS_OK)
    assert sizes(n_in, n_out, 100)[:2] == (libks.KS_ERR_UNSUPPORTED, libks.KS_ERR_UNSUPPORTED)
    assert sizes(n_in, n_out, 64)[:2] == (libks.KS_OK, libks.KS_OK)          # few rows: another launch
    ad = adapters(n_in, n_out)
    assert lib.ks_adapter_backward(ad, P["ids"], P["dY"], P["X"], P["H"], P["dX"], P["dA"], P["dB"], 100, libks.DTYPE_F32,
                                   P["ws"], 1 << 39, None) == libks.KS_ERR_UNSUPPORTED
    w = (ctypes.c_void_p * 1)(P["W"])
    assert lib.ks_chain_adapter_backward(libks._patterns([(1, n_out, n_in, 1)]), 1, w, None, ad, P["ids"], P["dY"], P["X"],
                                         P["H"], P["dX"], P["dA"], P["dB"], 100, libks.DTYPE_F32, P["ws"], 1 << 39,
                                         None) == libks.KS_ERR_UNSUPPORTED
