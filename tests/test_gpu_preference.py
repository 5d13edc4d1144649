"""Token log probabilities and the preference loss (needs an MI355X) against
the formulas in 64 bits.

Tolerances. l = (x - max) - log(sum) and only the sum is formed in fp32: terms
that count (x - max > -20, the rest is below 2e-9 of the sum) have an exponent
off by at most 20 log2(e) 2^-23 and an exponential off by 2 ulp, and the sum of
at most V / 2048 + 32 rounded partial sums: under 4e-6 + (V / 2048 + 32) 2^-24
of log(sum); l itself is rounded once (2^-24 |l|). Rewards add T of these. The
gradient's probabilities are off by the same relative amounts, its factor by
what the rewards' errors move it (its slope is at most beta^2 / (4 P)), and a
bf16 gradient is rounded once (2^-8 with margin for the one before it).
"""
from __future__ import annotations

import pytest
import torch
import torch.nn.functional as F

from gpu_helpers import DEV, require_gpu
from kronecker_sparse_structured_amd import layer, libks

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def formula(x, labels, ref=None, beta=0.1, e=0.0):
    x, labels = x.double().cpu(), labels.cpu()
    S, T, V = x.shape
    on = labels >= 0
    tokens = torch.zeros(S, T, dtype=torch.float64)
    for s in range(S):
        t = on[s].nonzero()[:, 0]
        tokens[s, t] = x[s, t, labels[s, t]] - torch.logsumexp(x[s, t], dim=1)
    out = {"tokens": tokens, "total": tokens.sum(1)}
    if ref is None:
        return out
    P = S // 2
    ratio = torch.where(on, tokens - torch.where(on, ref.double().cpu(), 0.0), 0.0)
    R = beta * ratio.sum(1)
    z = R[:P] - R[P:]
    out["rewards"] = R
    out["loss"] = ((1 - e) * F.softplus(-z) + e * F.softplus(z)).mean()
    c = beta * (e * torch.sigmoid(z) - (1 - e) * torch.sigmoid(-z)) / P
    d = torch.zeros(S, T, V, dtype=torch.float64)
    for s in range(S):
        t = on[s].nonzero()[:, 0]
        p = -torch.softmax(x[s, t], dim=1)
        p[torch.arange(len(t)), labels[s, t]] += 1
        d[s, t] = p * (c[s] if s < P else -c[s - P])
    out["d"] = d
    return out


def token_tol(V):
    return 4e-6 + (V / 2048 + 32) * 2.0 ** -24


def check(x, labels, ref, beta, e, got, want=None, upstream=1.0):
    loss, rewards, tokens, d = got
    want = want or formula(x, labels, ref, beta, e)
    S, T, V = x.shape
    P = S // 2
    tol = token_tol(V)
    err = (tokens.double().cpu() - want["tokens"]).abs()
    assert bool((err <= tol + 2.0 ** -23 * want["tokens"].abs()).all()), float(err.max())
    per = (tol + 2.0 ** -23 * want["tokens"].abs()).sum(1) * beta + 2.0 ** -23 * want["rewards"].abs()
    assert bool(((rewards.double().cpu() - want["rewards"]).abs() <= per).all())
    z = per[:P] + per[P:]
    assert abs(float(loss) - float(want["loss"])) <= float(z.mean()) + 2.0 ** -22 * float(want["loss"])
    if d is None:
        return
    c = (beta * z / (4 * P)).repeat(2)[:, None, None] * upstream
    scale = beta / P * upstream
    w = want["d"] * upstream
    bound = c + w.abs() * (2 * tol + 2.0 ** -21) + scale * 2.0 ** -40
    if d.dtype == BF16:
        bound = bound + w.abs() * 2.0 ** -8
    err = (d.double().cpu() - w).abs()
    assert bool((err <= bound).all()), float((err / bound).max())


def draw(P, T, V, dtype, seed, pad=0.3):
    g = torch.Generator().manual_seed(seed)
    x = (3 * torch.randn(2 * P, T, V, generator=g)).to(dtype).to(DEV)
    labels = torch.randint(V, (2 * P, T), generator=g)
    labels[torch.rand(2 * P, T, generator=g) < pad] = -100
    ref = -3 * torch.rand(2 * P, T, generator=g)
    return x, labels.to(DEV), ref.to(DEV)


CASES = [(1, 1, 1, F32), (1, 1, 7, BF16), (2, 3, 50, F32), (1, 17, 1000, BF16), (3, 5, 1001, F32), (2, 4, 4099, BF16),
         (1, 2, 32000, F32), (5, 3, 513, BF16), (1, 3, 50257, BF16), (1, 1, 262145, F32)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "%d-%d-%d-%s" % (*c[:3], str(c[3])[6:]))
@pytest.mark.parametrize("e", [0.0, 0.2])
def test_loss_and_gradient(case, e):
    require_gpu()
    P, T, V, dtype = case
    x, labels, ref = draw(P, T, V, dtype, seed=P * T + V)
    got = libks.preference_loss(x, labels, ref, beta=0.3, smoothing=e)
    check(x, labels, ref, 0.3, e, got)
    again = libks.preference_loss(x, labels, ref, beta=0.3, smoothing=e)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    total, tokens = libks.sequence_logp(x, labels)
    assert torch.equal(tokens, got[2])
    assert float((total.double() - tokens.double().sum(1)).abs().max()) <= 2.0 ** -23 * float(tokens.abs().sum())


def test_masked_rows_may_hold_anything():
    require_gpu()
    for dtype in (F32, BF16):
        x, labels, ref = draw(2, 6, 301, dtype, seed=3)
        labels[1] = -1                                  # a sequence without a token
        labels[2, :] = torch.arange(6, device=DEV)      # and one without a mask
        want = formula(x, labels, ref, 0.1, 0.0)
        x[labels < 0] = float("nan")
        ref[labels < 0] = float("inf")
        got = libks.preference_loss(x, labels, ref)
        check(x, labels, ref, 0.1, 0.0, got, want=want)
        assert not got[3][labels < 0].any() and not got[2][labels < 0].any()


def test_masked_vocabulary():
    require_gpu()
    for dtype in (F32, BF16):
        x, labels, ref = draw(1, 4, 1000, dtype, seed=5, pad=0.0)
        for low in (float("-inf"), torch.finfo(dtype).min):
            y = x.clone()
            y[:, :, 10:] = low
            labels.clamp_(max=9)
            check(y, labels, ref, 0.1, 0.0, libks.preference_loss(y, labels, ref))
        # nothing of the vocabulary left: uniform at the lowest value, not a number at -inf
        y[0, 0] = torch.finfo(dtype).min
        y[1, 0] = float("-inf")
        _, tokens = libks.sequence_logp(y, labels)
        assert abs(float(tokens[0, 0]) + float(torch.log(torch.tensor(1000.0)))) < 1e-5
        assert torch.isnan(tokens[1, 0]) and torch.isfinite(tokens[:, 1:]).all()
        # NaN and +inf in a row that counts are seen, and only there
        z = x.clone()
        z[0, 1, 3] = float("nan")
        z[1, 2, 3] = float("inf")
        _, tokens = libks.sequence_logp(z, labels)
        bad = torch.zeros_like(tokens, dtype=torch.bool)
        bad[0, 1] = bad[1, 2] = True
        assert torch.equal(torch.isnan(tokens), bad)


def test_label_outside_the_vocabulary_gives_nan():
    require_gpu()
    x, labels, ref = draw(1, 3, 40, F32, seed=1, pad=0.0)
    labels[0, 1] = 40
    loss, rewards, tokens, d = libks.preference_loss(x, labels, ref)
    assert torch.isnan(tokens[0, 1]) and torch.isnan(loss) and torch.isfinite(tokens[1]).all()


def test_strides_in_place_and_other_stream():
    require_gpu()
    for dtype, V in ((F32, 77), (BF16, 1003)):
        big, labels, ref = draw(2, 9, V, dtype, seed=7)
        x, lab, r = big[:, :-1], labels[:, 1:], ref[:, :-1]     # shifted by one, no copies
        want = formula(x, lab, r, 0.1, 0.1)
        check(x, lab, r, 0.1, 0.1, libks.preference_loss(x, lab, r, smoothing=0.1), want=want)
        wide = torch.zeros(4, 8, V + 5, dtype=dtype, device=DEV)
        d = wide[:, :, 2:2 + V]                                  # its rows start elsewhere in 16 bytes
        check(x, lab, r, 0.1, 0.1, libks.preference_loss(x, lab, r, smoothing=0.1, dlogits=d), want=want)
        assert not wide[:, :, :2].any() and not wide[:, :, 2 + V:].any()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        keep = big[:, -1].clone()
        with torch.cuda.stream(side):
            got = libks.preference_loss(x, lab, r, smoothing=0.1, dlogits=x)
        side.synchronize()
        check(torch.zeros_like(x), lab, r, 0.1, 0.1, got, want=want)
        assert torch.equal(big[:, -1], keep)                     # the cut-off position is not touched


def test_autograd_and_differences():
    require_gpu()
    x, labels, ref = draw(2, 5, 60, F32, seed=11)
    x.requires_grad_(True)
    loss, rewards, tokens = layer.preference_loss(x, labels, ref, beta=0.5, smoothing=0.1)
    (2.5 * loss).backward()
    check(x.detach(), labels, ref, 0.5, 0.1, (loss.detach(), rewards, tokens, x.grad), upstream=2.5)
    D = torch.randn(x.shape, generator=torch.Generator().manual_seed(2)).double()
    h = 1e-4
    up, down = (float(formula(x.detach().double().cpu() + s * h * D, labels, ref, 0.5, 0.1)["loss"]) for s in (1, -1))
    num = 2.5 * (up - down) / (2 * h)
    ana = float((x.grad.double().cpu() * D).sum())
    # fp32 gradient values (relative 1e-5 of sum |d| |D|) and the difference's own h^2
    assert abs(num - ana) <= 1e-5 * float((x.grad.double().cpu().abs() * D.abs()).sum()) + 1e-6


def test_no_pairs_and_no_tokens():
    require_gpu()
    none = torch.empty(0, 4, 10, device=DEV)
    loss, rewards, tokens, d = libks.preference_loss(none, torch.empty(0, 4, dtype=torch.int64, device=DEV),
                                                     torch.empty(0, 4, device=DEV))
    assert float(loss) == 0.0 and rewards.numel() == tokens.numel() == d.numel() == 0
    loss, rewards, tokens, d = libks.preference_loss(torch.empty(2, 0, 10, device=DEV),
                                                     torch.empty(2, 0, dtype=torch.int64, device=DEV),
                                                     torch.empty(2, 0, device=DEV))
    assert abs(float(loss) - 0.6931471805599453) < 1e-6 and not rewards.any()


def test_graph_replays():
    require_gpu()
    x, labels, ref = draw(2, 5, 500, BF16, seed=13)
    d = torch.empty_like(x)
    libks.preference_loss(x, labels, ref, dlogits=d)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, rewards, tokens, _ = libks.preference_loss(x, labels, ref, dlogits=d)
    for _ in range(4):
        x.normal_()
        want = libks.preference_loss(x, labels, ref)
        d.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, want[0]) and torch.equal(rewards, want[1]) and torch.equal(d, want[3])


def test_logits_past_2_31_elements():
    require_gpu()
    S, T, V = 2, 22_000, 50_257
    x = torch.empty(S, T, V, dtype=BF16, device=DEV)
    x.normal_(generator=torch.Generator(device=DEV).manual_seed(1))
    labels = torch.full((S, T), -1, dtype=torch.int64, device=DEV)
    rows = torch.tensor([0, 1, 11_111, T - 2, T - 1], device=DEV)
    labels[:, rows] = torch.randint(V, (S, 5), device=DEV, generator=torch.Generator(device=DEV).manual_seed(2))
    ref = torch.full((S, T), -11.0, device=DEV)
    loss, rewards, tokens, d = libks.preference_loss(x, labels, ref)
    want = formula(x[:, rows], labels[:, rows], ref[:, rows])
    check(x[:, rows], labels[:, rows], ref[:, rows], 0.1, 0.0, (loss, rewards, tokens[:, rows], d[:, rows]), want=want)
    assert not d[1, 11_112:T - 2].any()
