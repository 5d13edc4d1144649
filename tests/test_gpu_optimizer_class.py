"""The optimizer class (needs an MI355X): a step that is refused counts for
nothing."""
from __future__ import annotations

import pytest
import torch

from gpu_helpers import DEV, require_gpu
from kronecker_sparse_structured_amd import optim

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
def test_a_refused_step_is_not_counted(bits):
    require_gpu()

    def make():
        a, b = (torch.nn.Parameter(torch.full((40, 7), 0.5, device=DEV)) for _ in range(2))
        return a, b, optim.AdamW([{"params": [a]}, {"params": [b], "lr": 1e-2}], state_bits=bits, seed=3)

    a, b, opt = make()
    a.grad, b.grad = torch.ones_like(a), torch.ones_like(b)
    kept, b.data = b.data, torch.full((7, 40), 0.5, device=DEV).t()          # a layout that the kernels refuse
    with pytest.raises(ValueError):
        opt.step()
    assert all(s["step"] == 0 for s in opt.state.values()) and bool((a == 0.5).all())
    b.data = kept
    opt.step()
    a2, b2, fresh = make()
    a2.grad, b2.grad = torch.ones_like(a2), torch.ones_like(b2)
    fresh.step()
    assert torch.equal(a, a2) and torch.equal(b, b2)
    assert [s["step"] for s in opt.state.values()] == [s["step"] for s in fresh.state.values()] == [1, 1]
