"""Arguments of the optimizer's handle that the kernels read or write through
their address (needs an MI355X): a host tensor, a number or another type is
refused before a launch."""
from __future__ import annotations

import pytest
import torch

from gpu_helpers import DEV, require_gpu
from kronecker_sparse_structured_amd import libks

pytestmark = pytest.mark.gpu


def handle():
    return libks.AdamW(*([torch.ones(300, device=DEV)] for _ in range(4)))


BAD = {"host": lambda: torch.ones(()), "double": lambda: torch.ones((), dtype=torch.float64, device=DEV),
       "half": lambda: torch.ones((), dtype=torch.bfloat16, device=DEV), "none": lambda: torch.ones(0, device=DEV),
       "many": lambda: torch.ones(2, device=DEV), "number": lambda: 4096, "float": lambda: 1.5}


@pytest.mark.parametrize("bad", BAD)
def test_norm_that_cannot_be_read(bad):
    require_gpu()
    opt = handle()
    with pytest.raises(ValueError, match="norm"):
        opt.step(1, lr=0.1, max_norm=1.0, norm=BAD[bad]())
    with pytest.raises(ValueError, match="norm"):
        opt.step(1, lr=0.1, norm=BAD[bad]())
    with pytest.raises(ValueError, match="out"):
        opt.grad_norm(out=BAD[bad]())
    torch.cuda.synchronize()
    assert bool((opt._keep[0][0] == 1).all())


def test_norm_of_either_shape():
    require_gpu()
    for shape in ((), (1,)):
        opt, norm = handle(), torch.empty(shape, device=DEV)
        assert opt.grad_norm(out=norm) is norm and abs(float(norm) - 300 ** 0.5) < 1e-5
        assert opt.step(1, lr=0.1, max_norm=1.0, norm=norm) is norm
