"""Distillation (needs an MI355X): 64-bit ids of absent entries, whatever negative
number stands for them, beside a token that a row has more than once."""
from __future__ import annotations

import pytest
import torch

import test_gpu_distillation as dist
from gpu_helpers import require_gpu
from kronecker_sparse_structured_amd import layer, libks

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("none", [-1, -(1 << 31), -(1 << 32) + 5, -(1 << 63) + 5, -(1 << 63)])
def test_any_negative_id_is_no_entry(dtype, none):
    require_gpu()
    # its lower 32 bits are a token that follows it in the row
    token = none & 0xffffffff if none & 0xffffffff < 300 else 5
    x, labels, ids, top = dist.draw(2, 3, 300, 8, dtype, seed=21, pad=0.0, few=0.0, ids=torch.int64)
    ids[:, :, 0] = none
    ids[:, :, 3] = token
    ids[0, :, 5:7] = ids[0, :, 4:5]                   # a token more than once
    labels[1, 0] = token
    for w, T in ((1.0, 1.0), (0.6, 2.0)):
        want = dist.formula(x, labels, ids, top, w, T)
        dist.check(libks.distillation_loss(x, labels, ids, top, w, T), want)
        leaf = x.clone().requires_grad_(True)
        loss, tokens = layer.distillation_loss(leaf, labels, ids, top, w, T)
        loss.backward()
        dist.check((loss.detach(), tokens, leaf.grad), want)
