"""Distillation from a teacher's highest logits (needs an MI355X) against the
formulas in 64 bits.

Tolerances. Both sums of exponentials are formed as those of token log
probabilities: terms that count (x - max > -20 T, the rest is below 2e-9 of the
sum) have an exponent off by at most 20 log2(e) 2^-23 and an exponential off by 2
ulp, and the sum of at most V / 2048 + 32 rounded partial sums is off by tol =
4e-6 + (V / 2048 + 32) 2^-24 of itself, so log p by tol (it is settled in double).
The teacher's sum is one of 256 values at most: 4e-6 as well, for log q and,
relative, for q; log q is kept in fp32 (2^-24 of it). So with d_k = log q_k - log p_k
  token: w T^2 sum_k q_k (3 tol + 2^-23 |log q_k| + (tol + 2^-22) |d_k|)
         + (1 - w) tol + 2^-23 |token|
  dx:    (w T (p + q) + (1 - w) (p1 + 1[label])) (2 tol + 2^-20) / N
and a bf16 gradient is rounded once more (2^-8 of it, half a step).
"""
from __future__ import annotations

import math

import pytest
import torch

from gpu_helpers import DEV, require_gpu
from kronecker_sparse_structured_amd import libks

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def formula(x, labels, ids, top, w, T):
    """(loss, tokens, dx) and their bounds, row by row in 64 bits on the CPU."""
    x, labels, ids, top = x.double().cpu(), labels.cpu(), ids.cpu().long(), top.double().cpu()
    S, n, V = x.shape
    tol = 4e-6 + (V / 2048 + 32) * 2.0 ** -24
    tokens, et = torch.zeros(S, n, dtype=torch.float64), torch.zeros(S, n, dtype=torch.float64)
    dx, ed = torch.zeros(S, n, V, dtype=torch.float64), torch.zeros(S, n, V, dtype=torch.float64)
    N = max(int((labels >= 0).sum()), 1)
    for s in range(S):
        for t in range(n):
            if labels[s, t] < 0:
                continue
            r = x[s, t]
            logp, logp1 = torch.log_softmax(r / T, 0), torch.log_softmax(r, 0)
            have = (ids[s, t] >= 0) & (top[s, t] > -math.inf)
            k, g, size = ids[s, t][have], torch.zeros(V, dtype=torch.float64), torch.zeros(V, dtype=torch.float64)
            if w > 0 and len(k):
                logq = torch.log_softmax(top[s, t][have] / T, 0)
                q, d = logq.exp(), logq - logp[k]
                tokens[s, t] += w * T * T * float((q * d)[q > 0].sum())
                et[s, t] += w * T * T * float((q * (3 * tol + 2.0 ** -23 * logq.abs()
                                                    + (tol + 2.0 ** -22) * d.abs()))[q > 0].sum())
                g += w * T * logp.exp()
                size += w * T * logp.exp()
                g.index_add_(0, k, -w * T * q)
                size.index_add_(0, k, w * T * q)
            if w < 1:
                tokens[s, t] -= (1 - w) * float(logp1[labels[s, t]])
                et[s, t] += (1 - w) * tol
                g += (1 - w) * logp1.exp()
                g[labels[s, t]] -= 1 - w
                size += (1 - w) * logp1.exp()
                size[labels[s, t]] += 1 - w
            et[s, t] += 2.0 ** -23 * abs(float(tokens[s, t]))
            dx[s, t], ed[s, t] = g / N, size * (2 * tol + 2.0 ** -20) / N
    loss = float(tokens.sum()) / N
    return (loss, tokens, dx), (float(et.sum()) / N + 2.0 ** -23 * abs(loss), et, ed)


def check(got, want, upstream=1.0):
    (loss, tokens, dx), (el, et, ed) = want
    assert abs(float(got[0]) - loss) <= el, (float(got[0]), loss, el)
    err = (got[1].double().cpu() - tokens).abs()
    assert bool((err <= et).all()), float((err / et.clamp(min=1e-30)).max())
    if got[2] is None:
        return
    bound = ed * upstream + 1e-30
    if got[2].dtype == BF16:
        bound = bound * (1 + 2.0 ** -7) + dx.abs() * upstream * 2.0 ** -8
    err = (got[2].double().cpu() - dx * upstream).abs()
    assert bool((err <= bound).all()), float((err / bound).max())


def draw(S, T, V, K, dtype, seed, pad=0.3, few=0.3, top=F32, ids=torch.int32):
    g = torch.Generator().manual_seed(seed)
    x = 2 * torch.randn(S, T, V, generator=g)
    teacher, at = (x + torch.randn(S, T, V, generator=g)).topk(min(K, V), dim=2)
    if K > V:                                        # the same tokens more than once
        teacher, at = torch.cat([teacher] * (K // V + 1), 2)[:, :, :K], torch.cat([at] * (K // V + 1), 2)[:, :, :K]
    cut = torch.rand(S, T, K, generator=g) < few
    cut[:, :, 0] = False
    at = torch.where(cut, torch.full_like(at, -1), at)
    labels = torch.randint(V, (S, T), generator=g)
    labels[torch.rand(S, T, generator=g) < 0.5] = at[:, :, 0][torch.rand(S, T, generator=g) < 2][0]
    labels[torch.rand(S, T, generator=g) < pad] = -100
    return x.to(dtype).to(DEV), labels.to(DEV), at.to(ids).to(DEV).contiguous(), teacher.to(top).to(DEV).contiguous()


CASES = [(1, 1, 1, 1, F32), (1, 1, 7, 3, BF16), (2, 3, 50, 50, F32), (1, 17, 1000, 64, BF16), (3, 5, 1001, 5, F32),
         (2, 4, 4099, 256, BF16), (1, 2, 32000, 100, F32), (5, 3, 513, 1, BF16), (1, 3, 50257, 64, BF16),
         (1, 2, 50257, 33, F32), (1, 1, 131077, 8, BF16), (1, 1, 262145, 17, F32), (1, 2, 5, 40, F32)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "%d-%d-%d-%d-%s" % (*c[:4], str(c[4])[6:]))
@pytest.mark.parametrize("w,T", [(1.0, 1.0), (0.7, 1.0), (0.5, 2.5), (1.0, 0.5), (0.0, 1.0), (0.0, 3.0)])
def test_loss_and_gradient(case, w, T):
    require_gpu()
    S, n, V, K, dtype = case
    data = draw(S, n, V, K, dtype, seed=S * n + V + K)
    want = formula(*data, w, T)
    got = libks.distillation_loss(*data, weight=w, temperature=T)
    check(got, want)
    again = libks.distillation_loss(*data, weight=w, temperature=T)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    loss, tokens, none = libks.distillation_loss(*data, weight=w, temperature=T, grad=False)
    assert none is None
    check((loss, tokens, None), want)


@pytest.mark.parametrize("top", [F32, BF16])
@pytest.mark.parametrize("ids", [torch.int32, torch.int64])
def test_types_of_the_teacher(top, ids):
    require_gpu()
    data = draw(2, 5, 300, 20, BF16, seed=1, top=top, ids=ids)
    check(libks.distillation_loss(*data, weight=0.6, temperature=2.0), formula(*data, 0.6, 2.0))


def test_masked_rows_may_hold_anything():
    require_gpu()
    for dtype in (F32, BF16):
        x, labels, ids, top = draw(2, 6, 301, 9, dtype, seed=3)
        labels[1] = -1
        want = formula(x, labels, ids, top, 0.5, 2.0)
        off = labels < 0
        x[off], top[off], ids[off] = float("nan"), float("inf"), 1 << 30
        got = libks.distillation_loss(x, labels, ids, top, weight=0.5, temperature=2.0)
        check(got, want)
        assert not got[2][off].any() and not got[1][off].any()
        labels.fill_(-1)                             # nothing is left
        loss, tokens, d = libks.distillation_loss(x, labels, ids, top, weight=0.5, temperature=2.0)
        assert float(loss) == 0.0 and not tokens.any() and not d.any()


def test_rows_without_entries_and_entries_without_weight():
    require_gpu()
    for dtype in (F32, BF16):
        x, labels, ids, top = draw(2, 4, 77, 6, dtype, seed=5, pad=0.0)
        ids[0, 0] = -1
        top[0, 1] = float("-inf")
        top[0, 2, 1:] = float("-inf")
        top[1, 0, 2] = torch.finfo(F32).min
        top[1, 1] = torch.finfo(F32).min              # equal, however low
        for w in (1.0, 0.4):
            check(libks.distillation_loss(x, labels, ids, top, weight=w, temperature=1.5),
                  formula(x, labels, ids, top, w, 1.5))


def test_the_same_token_twice():
    require_gpu()
    x, labels, ids, top = draw(1, 3, 64, 12, F32, seed=7, pad=0.0, few=0.0)
    ids[0, 0] = 5
    ids[0, 1, ::2] = 9
    ids[0, 2, 3:9] = ids[0, 2, 1]
    labels[0, 0], labels[0, 1] = 5, 9
    got = libks.distillation_loss(x, labels, ids, top, weight=0.5, temperature=2.0)
    check(got, formula(x, labels, ids, top, 0.5, 2.0))
    for _ in range(5):
        assert torch.equal(libks.distillation_loss(x, labels, ids, top, weight=0.5, temperature=2.0)[2], got[2])


def test_masked_vocabulary():
    require_gpu()
    for dtype in (F32, BF16):
        x, labels, ids, top = draw(1, 4, 1000, 8, dtype, seed=5, pad=0.0)
        labels.clamp_(max=9)
        ids.clamp_(max=9)
        for low in (float("-inf"), torch.finfo(dtype).min):
            y = x.clone()
            y[:, :, 10:] = low
            for w, T in ((1.0, 1.0), (0.5, 2.0)):
                check(libks.distillation_loss(y, labels, ids, top, weight=w, temperature=T),
                      formula(y, labels, ids, top, w, T))
        # the teacher wants what the student cannot give
        y[0, 0, 3] = float("-inf")
        ids[0, 0, 0] = 3
        _, tokens, _ = libks.distillation_loss(y, labels, ids, top)
        assert float(tokens[0, 0]) == math.inf and torch.isfinite(tokens[0, 1:]).all()
        # NaN and +inf are seen in their rows, and only there
        z = x.clone()
        z[0, 1, 3] = float("nan")
        z[0, 2, 3] = float("inf")
        _, tokens, d = libks.distillation_loss(z, labels, ids, top, weight=0.5, temperature=2.0)
        assert torch.isnan(tokens).tolist() == [[False, True, True, False]]
        assert torch.isnan(d[0, 1]).all() and torch.isnan(d[0, 2]).any() and torch.isfinite(d[0, [0, 3]]).all()
        top[0, 3, 0] = float("nan")
        _, tokens, d = libks.distillation_loss(x, labels, ids, top)
        assert torch.isnan(tokens).tolist() == [[False, False, False, True]] and torch.isnan(d[0, 3]).any()


def test_tokens_outside_the_vocabulary_give_nan():
    require_gpu()
    x, labels, ids, top = draw(1, 3, 40, 4, F32, seed=1, pad=0.0, few=0.0)
    ids[0, 1, 2] = 40
    loss, tokens, d = libks.distillation_loss(x, labels, ids, top)
    assert torch.isnan(tokens).tolist() == [[False, True, False]] and torch.isnan(d[0, 1]).any() and torch.isnan(loss)
    wide = ids.long()
    wide[0, 1, 2] = 1 << 40
    assert torch.isnan(libks.distillation_loss(x, labels, wide, top)[1]).tolist() == [[False, True, False]]
    ids[0, 1, 2] = 3
    labels[0, 2] = 40
    assert torch.isnan(libks.distillation_loss(x, labels, ids, top, weight=0.5)[1]).tolist() == [[False, False, True]]
    # with weight 1 a label only says that its position counts
    check(libks.distillation_loss(x, labels, ids, top), formula(x, labels.clamp(max=39), ids, top, 1.0, 1.0))


def test_strides_in_place_and_other_stream():
    require_gpu()
    for dtype, V in ((F32, 77), (BF16, 1003), (BF16, 60001)):
        big, labels, ids, top = draw(2, 5, V, 12, dtype, seed=7)
        x, lab, k, t = big[:, :-1], labels[:, 1:], ids[:, :-1, :7], top[:, :-1, :7]      # no copies
        want = formula(x, lab, k, t, 0.5, 2.0)
        check(libks.distillation_loss(x, lab, k, t, 0.5, 2.0), want)
        wide = torch.zeros(2, 4, V + 5, dtype=dtype, device=DEV)
        d = wide[:, :, 2:2 + V]                                  # its rows start elsewhere in 16 bytes
        check(libks.distillation_loss(x, lab, k, t, 0.5, 2.0, dlogits=d), want)
        assert not wide[:, :, :2].any() and not wide[:, :, 2 + V:].any()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        keep = big[:, -1].clone()
        got = libks.distillation_loss(x, lab, k, t, 0.5, 2.0, dlogits=x, stream=side)
        side.synchronize()
        check(got, want)
        assert torch.equal(big[:, -1], keep)                     # the cut-off position is not touched


def test_no_rows():
    require_gpu()
    for S, T in ((0, 4), (2, 0)):
        loss, tokens, d = libks.distillation_loss(
            torch.empty(S, T, 10, device=DEV), torch.empty(S, T, dtype=torch.int64, device=DEV),
            torch.empty(S, T, 3, dtype=torch.int32, device=DEV), torch.empty(S, T, 3, device=DEV))
        assert float(loss) == 0.0 and tokens.shape == (S, T) and d.shape == (S, T, 10)


def test_graph_replays():
    require_gpu()
    x, labels, ids, top = draw(2, 5, 500, 16, BF16, seed=13)
    d = torch.empty_like(x)
    args = dict(weight=0.5, temperature=2.0, dlogits=d)
    libks.distillation_loss(x, labels, ids, top, **args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, tokens, _ = libks.distillation_loss(x, labels, ids, top, **args)
    for k in range(4):
        x.normal_()
        labels[0, k] = -labels[0, k] - 1
        want = libks.distillation_loss(x, labels, ids, top, weight=0.5, temperature=2.0)
        d.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, want[0]) and torch.equal(tokens, want[1]) and torch.equal(d, want[2])


def test_many_rows():
    """More rows than one launch of a workgroup a row counts by itself."""
    require_gpu()
    g = torch.Generator(device=DEV).manual_seed(1)
    S, T, V = 3, 3001, 33
    x = torch.randn(S, T, V, device=DEV, generator=g)
    labels = torch.randint(-9, V, (S, T), device=DEV, generator=g)
    top, ids = torch.randn(S, T, V, device=DEV, generator=g).topk(4, dim=2)
    loss, tokens, d = libks.distillation_loss(x, labels, ids, top, 0.5, 2.0)
    on = labels >= 0
    rows = on.nonzero()[::1000]
    some = (x[rows[:, 0], rows[:, 1]][None], labels[rows[:, 0], rows[:, 1]][None], ids[rows[:, 0], rows[:, 1]][None],
            top[rows[:, 0], rows[:, 1]][None])
    (_, want, dx), (_, et, ed) = formula(*some, 0.5, 2.0)
    share = len(rows) / float(on.sum())
    assert bool(((tokens[rows[:, 0], rows[:, 1]].double().cpu() - want[0]).abs() <= et[0]).all())
    assert bool(((d[rows[:, 0], rows[:, 1]].double().cpu() - dx[0] * share).abs() <= ed[0] * share + 1e-30).all())
    mean = float(tokens.double().sum()) / int(on.sum())
    assert abs(float(loss) - mean) <= 2.0 ** -22 * abs(mean)
    assert not d[~on].any()


def test_logits_past_2_31_elements():
    require_gpu()
    S, T, V = 2, 22_000, 50_257
    x = torch.empty(S, T, V, dtype=BF16, device=DEV)
    x.normal_(generator=torch.Generator(device=DEV).manual_seed(1))
    labels = torch.full((S, T), -1, dtype=torch.int64, device=DEV)
    rows = torch.tensor([0, 11_111, T - 1], device=DEV)
    g = torch.Generator(device=DEV).manual_seed(2)
    labels[:, rows] = torch.randint(V, (S, 3), device=DEV, generator=g)
    top, ids = torch.randn(S, T, 5, device=DEV, generator=g), torch.randint(V, (S, T, 5), device=DEV, generator=g)
    loss, tokens, d = libks.distillation_loss(x, labels, ids, top, 0.5, 2.0, dlogits=x.clone())
    want = formula(x[:, rows], labels[:, rows], ids[:, rows], top[:, rows], 0.5, 2.0)
    check((loss, tokens[:, rows], libks.distillation_loss(x, labels, ids, top, 0.5, 2.0)[2][:, rows]), want)
    assert not d[1, 11_112:T - 1].any()


def test_refusals():
    require_gpu()
    x, labels, ids, top = draw(1, 2, 20, 4, F32, seed=1)
    bad = [(x[0], labels, ids, top), (x, labels.int(), ids, top), (x, labels, ids[:, :1], top), (x, labels, ids.short(), top),
           (x, labels, ids, top.double()), (x, labels, ids, top[:, :, :3]), (x, labels, ids.cpu(), top),
           (x.half(), labels, ids, top), (x, labels, ids.transpose(1, 2).contiguous().transpose(1, 2), top)]
    for args in bad:
        with pytest.raises((ValueError, TypeError)):
            libks.distillation_loss(*args)
    for kw in (dict(dlogits=x.bfloat16()), dict(dlogits=torch.empty_like(x), grad=False)):
        with pytest.raises((ValueError, TypeError)):
            libks.distillation_loss(x, labels, ids, top, **kw)
    for kw in (dict(weight=1.5), dict(temperature=0.0), dict(temperature=-1.0)):
        with pytest.raises(libks.KSError):
            libks.distillation_loss(x, labels, ids, top, **kw)
    many = torch.zeros(1, 2, 257, dtype=torch.int32, device=DEV)
    with pytest.raises(libks.KSError):
        libks.distillation_loss(x, labels, many, many.float())
