"""The clip of the AdamW step (needs an MI355X): a bound above the norm leaves
every bit of a step without one."""
from __future__ import annotations

import pytest
import torch

from gpu_helpers import DEV, require_gpu
from kronecker_sparse_structured_amd import libks

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bits", [32, 8])
def test_a_bound_above_the_norm_clips_nothing(bits, gt):
    require_gpu()
    sizes = [5, 256, 4097, 70001]
    done = []
    for max_norm in (None, 1e9):
        g = torch.Generator().manual_seed(8)
        ps = [torch.randn(n, generator=g).to(DEV) for n in sizes]
        gs = [(0.05 * torch.randn(n, generator=g)).to(gt).to(DEV) for n in sizes]
        if bits == 32:
            ms = [(0.01 * torch.randn(n, generator=g)).to(DEV) for n in sizes]
            vs = [(1e-3 * torch.rand(n, generator=g)).to(DEV) for n in sizes]
            scales = None
        else:
            ms = [torch.randint(-127, 128, (n,), generator=g).to(torch.int8).to(DEV) for n in sizes]
            vs = [torch.randint(0, 256, (n,), generator=g).to(torch.uint8).to(DEV) for n in sizes]
            scales = [torch.full((-(-n // 256), 2), 1e-3, device=DEV) for n in sizes]
        norm = libks.AdamW(ps, gs, ms, vs, scales).step(2, lr=2e-3, max_norm=max_norm, seed=5)
        assert max_norm is None or 1.0 < float(norm) < 1e9
        done.append([*ps, *ms, *vs, *(scales or ())])
    assert all(torch.equal(x, y) for x, y in zip(*done))
    assert any((t != 0).any() for t in done[0])
