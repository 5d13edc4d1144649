"""Distillation over more positions than each workgroup counts by itself, and the
kernels that only such batches reach (needs an MI355X).

Few of the positions count, so the formula in 64 bits is formed of those alone: it
is theirs whatever the others are. The bounds are those of the small batches: a
lane adds a vector's values (8 at most), 16 vectors, two values beside them, and up
to 9 exchanges follow, which is no more than the V / 2048 + 32 partial sums that they
count. A token stands in a row up to 4 times, 3 roundings more in the sum of its
entries, among the 16 that the gradient's bound has room for."""
from __future__ import annotations

import pytest
import torch

import test_gpu_distillation as dist
from gpu_helpers import DEV, require_gpu
from kronecker_sparse_structured_amd import layer, libks

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
MODES = [(1.0, 1.0), (0.7, 1.0), (0.5, 2.0), (0.5, 2.5)]


def draw(S, T, V, K, dtype, seed):
    """(data, the positions that count)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.empty(S, T, V, dtype=dtype, device=DEV).normal_(generator=g)
    n = S * T
    rows = torch.tensor([0, 1, 63, 64, n // 2, n // 2 + 1, n - 1], device=DEV)
    flat = x.view(n, V)[rows].float()
    top = torch.randn(n, K, device=DEV, generator=g)
    ids = torch.randint(V, (n, K), device=DEV, generator=g)
    top[rows], ids[rows] = (flat + torch.randn(len(rows), V, device=DEV, generator=g)).topk(K, dim=1)
    # a token again 64, 128 and 192 entries later; a row with fewer entries; one with none
    for r in rows[1:4]:
        for by in (64, 128, 192):
            if K > by:
                some = min(5, K - by)
                ids[r, by:by + some] = ids[r, :some]
    ids[rows[4], K // 3:] = -1
    ids[rows[5]] = -1
    labels = torch.full((n,), -100, dtype=torch.int64, device=DEV)
    labels[rows] = torch.randint(V, (len(rows),), device=DEV, generator=g)
    labels[rows[:4]] = ids[rows[:4], 0]               # a token that the teacher has, in three of them again later
    labels[rows[6]] = V - 1
    return (x, labels.view(S, T), ids.view(S, T, K).to(torch.int32), top.view(S, T, K)), rows


def check(got, data, rows, w, T, upstream=1.0):
    x, labels, ids, top = data
    V, K = x.shape[2], ids.shape[2]

    def pick(t, *last):
        return t.reshape(-1, *last)[rows][None]

    want = dist.formula(pick(x, V), pick(labels), pick(ids, K), pick(top, K), w, T)
    loss, tokens, d = got
    dist.check((loss, pick(tokens), None if d is None else pick(d, V)), want, upstream)
    off = (labels < 0).view(-1)
    assert not tokens.reshape(-1)[off].any()
    if d is not None:
        assert not d.reshape(-1, V)[off].any()


# vocabularies that each of the kernels which hold a row has, from one wave to 16, and longer ones
CASES = [(40, 40, F32), (2000, 65, F32), (4001, 128, F32), (8003, 256, F32), (16001, 65, F32), (32002, 200, F32),
         (65001, 256, F32), (70001, 256, F32), (97, 65, BF16), (4001, 256, BF16), (8001, 200, BF16),
         (16003, 128, BF16), (32001, 65, BF16), (65001, 256, BF16), (131001, 64, BF16), (140001, 128, BF16)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "%d-%d-%s" % (*c[:2], str(c[2])[6:]))
def test_many_positions(case):
    require_gpu()
    V, K, dtype = case
    data, rows = draw(3, 701, V, K, dtype, seed=V + K)
    for w, T in MODES:
        got = libks.distillation_loss(*data, weight=w, temperature=T)
        check(got, data, rows, w, T)
        again = libks.distillation_loss(*data, weight=w, temperature=T)
        assert all(torch.equal(a, b) for a, b in zip(got, again))
        check(libks.distillation_loss(*data, weight=w, temperature=T, grad=False), data, rows, w, T)
        x = data[0].detach().requires_grad_(True)
        loss, tokens = layer.distillation_loss(x, *data[1:], w, T)
        (2.5 * loss).backward()
        check((loss.detach(), tokens, x.grad), data, rows, w, T, upstream=2.5)


@pytest.mark.parametrize("case", dist.CASES, ids=lambda c: "%d-%d-%d-%d-%s" % (*c[:4], str(c[4])[6:]))
def test_few_positions_at_temperature_2(case):
    require_gpu()
    S, n, V, K, dtype = case
    data = dist.draw(S, n, V, K, dtype, seed=S * n + V + K)
    own = torch.rand(S, n, generator=torch.Generator().manual_seed(V)) < 0.5
    labels = torch.where(own.to(DEV) & (data[1] >= 0), data[2][:, :, 0].long(), data[1])   # the row's own first entry
    data = (data[0], labels, *data[2:])
    for w, T in ((0.5, 2.0), (0.7, 1.0)):
        want = dist.formula(*data, w, T)
        dist.check(libks.distillation_loss(*data, weight=w, temperature=T), want)
        loss, tokens, _ = libks.distillation_loss(*data, weight=w, temperature=T, grad=False)
        dist.check((loss, tokens, None), want)
        x = data[0].detach().requires_grad_(True)
        loss, tokens = layer.distillation_loss(x, *data[1:], w, T)
        (2.5 * loss).backward()
        dist.check((loss.detach(), tokens, x.grad), want, upstream=2.5)


@pytest.mark.parametrize("case", [(70001, 256, F32), (140001, 128, BF16), (32001, 200, BF16)], ids=lambda c: "%d-%d-%s" % (*c[:2], str(c[2])[6:]))
def test_the_gradient_in_the_logits_place(case):
    """Also of rows that are read twice, in one call and with the gradient in a call of its own."""
    require_gpu()
    V, K, dtype = case
    data, rows = draw(3, 701, V, K, dtype, seed=V)
    for w, T in MODES:
        x = data[0].clone()
        loss, tokens, d = libks.distillation_loss(x, *data[1:], w, T, dlogits=x)
        assert d is x
        check((loss, tokens, d), data, rows, w, T)
        x = data[0].clone()
        loss, tokens, stats, _ = libks._distil_forward(x, *data[1:], w, T)
        want = libks._distil_backward(x, *data[1:], w, T, stats, None)
        lib, logits = libks.load(), libks._logits(x, data[1])
        status = lib.ks_distil_backward(logits, libks._teacher(*data[2:], x), w, T, stats.data_ptr(), None, x.data_ptr(),
                                        *libks._layout(x, "x"), libks._raw_stream(x.get_device()))
        assert status == libks.KS_OK and torch.equal(x, want)
