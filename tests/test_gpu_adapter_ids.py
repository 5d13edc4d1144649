"""Rows without an adapter (needs an MI355X): any id outside [0, count) means
none, on every path, and below -1 exactly what -1 means.

Tolerances as for the other adapter tests: sums of k fp32 terms within
k 2^-23 of the same sum of magnitudes.
"""
from __future__ import annotations

import itertools

import pytest
import torch

import oracle
from gpu_helpers import DEV, require_gpu
from kronecker_sparse_structured_amd import libks
from test_gpu_adapters import BF16, F32, PAIR, draw, formula, near

pytestmark = pytest.mark.gpu
LOW = -2 ** 31


def groups(count):
    """Every group of four rows over these ids, and a last group of three."""
    ids = list(itertools.chain(*itertools.product([LOW, -2, -1, 0, count - 1, count + 7], repeat=4)))
    return torch.tensor(ids + [LOW, -1, 1], dtype=torch.int32, device=DEV)


def as_none(ids, count):
    return torch.where((ids < 0) | (ids >= count), torch.full_like(ids, -1), ids)


@pytest.mark.parametrize("rank", [16, 20])
def test_groups_of_the_pair(rank):
    require_gpu()
    ids = groups(3)
    batch = ids.numel()
    X, A, B, scale, _ = draw(batch, 1024, 4096, 3, rank, BF16, BF16, seed=rank)
    Ws = [(torch.randn(a, d, b, c) / c ** 0.5).to(BF16).to(DEV) for a, b, c, d in PAIR]
    chain = libks.AdapterChain(Ws, PAIR, A, B, scale)
    dY = torch.randn(batch, 4096, device=DEV)
    Y, H = chain.matmul(X, ids, keep=True)
    same = chain.matmul(X, as_none(ids, 3), keep=True)
    assert torch.equal(Y, same[0]) and torch.equal(H, same[1])
    ref = formula(X, A, B, scale, ids)
    mag = formula(X.abs(), A.abs(), B.abs(), scale, ids)
    near(H, ref["H"], mag["H"], 1024 + 2, "H")
    Wn, x = [w.double().cpu().numpy() for w in Ws], X.double().cpu().numpy()
    base = torch.from_numpy(oracle.ks_chain_matmul(PAIR, Wn, x))
    size = torch.from_numpy(oracle.ks_chain_matmul(PAIR, [abs(w) for w in Wn], abs(x)))
    near(Y, base + ref["D"], size + mag["D"], 1024 + rank + 26 + 4, "Y")
    for got, want in zip(chain.backward(dY, X, H, ids), chain.backward(dY, X, H, as_none(ids, 3))):
        assert torch.equal(got, want)


@pytest.mark.parametrize("batch,xt,wt", [(9, F32, F32), (64, BF16, BF16), (128, F32, BF16), (1000, F32, F32),
                                         (4096, BF16, BF16), (5187, F32, BF16)])
def test_other_paths(batch, xt, wt):
    require_gpu()
    X, A, B, scale, _ = draw(batch, 64, 96, 3, 8, xt, wt, seed=batch)
    ids = groups(3)[-batch:].contiguous()
    none = as_none(ids, 3)
    dY = torch.randn(batch, 96, device=DEV)
    res = []
    for who in (ids, none):
        out, dX = torch.zeros(batch, 96, device=DEV), torch.zeros(batch, 64, device=DEV)
        _, H = libks.adapter_matmul(X, A, B, scale, who, out, keep=True)
        res.append((out, H, dX, *libks.adapter_backward(dY, X, H, A, B, scale, who, dX=dX)))
    assert all(torch.equal(a, b) for a, b in zip(*res))
    off = none < 0
    assert not any(t[off].any() for t in res[0][:3]) and res[0][0][~off].any(dim=1).all()
