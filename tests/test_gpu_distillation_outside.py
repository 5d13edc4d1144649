"""Distillation (needs an MI355X): a teacher's token or a label outside the
vocabulary makes its position's loss and whole gradient NaN, whatever else the row
holds, and leaves the others' as the formula has them."""
from __future__ import annotations

import pytest
import torch

import test_gpu_distillation as dist
from gpu_helpers import DEV, require_gpu
from kronecker_sparse_structured_amd import layer, libks

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
K = 100


def draw(S, T, V, dtype, seed):
    """Rows of entries that all have token 0 among them, in the first wave and later."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(S, T, V, device=DEV, generator=g).to(dtype)
    top = torch.randn(S, T, K, device=DEV, generator=g)
    ids = torch.randint(1, V, (S, T, K), device=DEV, generator=g, dtype=torch.int32)
    labels = torch.randint(1, V, (S, T), device=DEV, generator=g)
    ids[0, 0, :2] = torch.tensor([0, V])             # beside each other
    ids[0, 1, 1], ids[0, 1, 90] = V, 0               # in two waves
    ids[0, 2, 90], ids[0, 2, 0] = 1 << 30, 0
    ids[0, 3, 80], labels[0, 3] = 0, V               # of the label
    labels[0, 4], ids[0, 4, 3] = 0, V + 7            # no entry of token 0, but the label
    ids[0, 5, 0] = 0                                 # sound
    return x, labels, ids, top


# a row in registers, of few positions and of many, and longer ones
@pytest.mark.parametrize("case", [(1, 6, 300, F32), (1, 6, 50257, BF16), (350, 6, 300, F32), (350, 6, 9001, BF16),
                                  (1, 6, 70001, F32), (1, 6, 262145, BF16)], ids=lambda c: "%d-%d-%d-%s" % (*c[:3], str(c[3])[6:]))
def test_rows_with_tokens_outside_are_nan(case):
    require_gpu()
    S, T, V, dtype = case
    data = draw(S, T, V, dtype, seed=V)
    bad = torch.tensor([True, True, True, True, True, False], device=DEV)
    for w, temperature in ((0.5, 2.0), (0.6, 1.0), (0.5, 2.5), (1.0, 1.0)):
        if w == 1.0:
            bad[3] = False                           # a label only says that its position counts
        got = [libks.distillation_loss(*data, weight=w, temperature=temperature)]
        x = data[0].detach().requires_grad_(True)
        loss, tokens = layer.distillation_loss(x, *data[1:], w, temperature)
        loss.backward()
        got.append((loss.detach(), tokens, x.grad))
        for loss, tokens, d in got:
            assert torch.isnan(loss)
            assert torch.equal(torch.isnan(tokens[0]), bad) and torch.isfinite(tokens[1:]).all()
            assert torch.isnan(d[0, bad]).all()
            assert torch.isfinite(d[0, ~bad]).all() and torch.isfinite(d[1:]).all()
            share = 1.0 / (S * T)
            rows = (~bad).nonzero()[:, 0]
            one = tuple(t[:1, rows] for t in data)
            one = (one[0], one[1].clamp(max=V - 1), *one[2:])
            (_, want, dx), (_, et, ed) = dist.formula(*one, w, temperature)
            n = share * len(rows)                    # of the mean over all positions
            assert bool(((tokens[:1, rows].double().cpu() - want).abs() <= et).all())
            bound = ed * n + 1e-30
            if dtype == BF16:
                bound = bound * (1 + 2.0 ** -7) + dx.abs() * n * 2.0 ** -8
            assert bool(((d[:1, rows].double().cpu() - dx * n).abs() <= bound).all())
