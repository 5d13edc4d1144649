"""Beam selection and the reordering of states (needs an MI355X) against a plain
search in 64 bits.

The choices are whole numbers and have to be the plain ones wherever the ranks of
two candidates differ by more than a score can be off: a row's sum of
exponentials is formed like those of token log probabilities (terms off by
20 log2(e) 2^-23 and 2 ulp, 40 roundings of partial sums, then double), so a score
by tol = 4e-6 + 40 2^-24, and a score's output by 2^-24 of it more. Candidates of
one beam are ordered exactly, by logit and then token.
"""
from __future__ import annotations

import math

import pytest
import torch

from gpu_helpers import DEV, require_gpu
from kronecker_sparse_structured_amd import libks

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
TOL = 4e-6 + 40 * 2.0 ** -24


def candidates(x, scores, done, lengths, eos, penalty):
    """Of each request, (rank, flat, score, length) of every candidate, best first."""
    x, scores = x.double().cpu(), scores.double().cpu()
    R, W, V = x.shape
    out = []
    for r in range(R):
        found = []
        for w in range(W):
            s = float(scores[r, w])
            n = int(lengths[r, w]) if lengths is not None else 0
            if not math.isfinite(s):
                continue
            if done is not None and bool(done[r, w]):
                found.append((s / max(n, 1) ** penalty, w * V + eos, s, n))
                continue
            row = x[r, w]
            if bool(torch.isnan(row).any()) or bool((row == math.inf).any()) or bool((row == -math.inf).all()):
                continue
            value = s + row - torch.logsumexp(row, 0)
            best = torch.sort(value, descending=True, stable=True)
            for v, t in zip(best[0][:300].tolist(), best[1][:300].tolist()):
                if v > -math.inf:
                    found.append((v / max(n + 1, 1) ** penalty, w * V + t, v, n + 1))
        found.sort(key=lambda c: (-c[0], c[1]))
        out.append(found)
    return out


def check(x, scores, out_beams, done, lengths, eos, penalty, got, exact=True):
    R, W, V = x.shape
    want = candidates(x, scores, done, lengths, eos, penalty)
    b = libks.Beams(*(None if t is None else t.cpu() for t in got))
    assert b.scores.shape == (R, out_beams)
    for r in range(R):
        by_flat = {c[1]: c for c in want[r]}
        for j in range(out_beams):
            if j >= len(want[r]):
                assert float(b.scores[r, j]) == -math.inf and int(b.parents[r, j]) == 0
                assert int(b.tokens[r, j]) == (eos if eos is not None else 0)
                assert b.done is None or bool(b.done[r, j])
                assert b.lengths is None or int(b.lengths[r, j]) == 0
                continue
            flat = int(b.parents[r, j]) * V + int(b.tokens[r, j])
            rank, place, score, n = want[r][j]
            if exact:
                assert flat == place, (r, j, flat, place)
            else:       # as good as the plain choice
                assert abs(by_flat[flat][0] - rank) <= 2 * TOL, (r, j)
            _, _, score, n = by_flat[flat]
            assert abs(float(b.scores[r, j]) - score) <= TOL + 2.0 ** -23 * abs(score)
            assert b.done is None or bool(b.done[r, j]) == (int(b.tokens[r, j]) == eos)
            assert b.lengths is None or int(b.lengths[r, j]) == n
        flats = [int(b.parents[r, j]) * V + int(b.tokens[r, j]) for j in range(min(out_beams, len(want[r])))]
        assert len(set(flats)) == len(flats)


def draw(R, W, V, dtype, seed, ended=0.2):
    g = torch.Generator().manual_seed(seed)
    x = (3 * torch.randn(R, W, V, generator=g)).to(dtype).to(DEV)
    lengths = torch.randint(0, 30, (R, W), generator=g, dtype=torch.int32).to(DEV)
    scores = (-3 * torch.rand(R, W, generator=g)).to(DEV)
    done = (torch.rand(R, W, generator=g) < ended).to(DEV)
    return x, scores, done, lengths


def gaps(x, scores, done, lengths, eos, penalty, n):
    """Whether the n + 1 best ranks of every request lie further apart than scores can be off."""
    for found in candidates(x, scores, done, lengths, eos, penalty):
        ranks = [c[0] for c in found[:n + 1]]
        flats = [c[1] // x.shape[2] for c in found[:n + 1]]
        for a, b, p, q in zip(ranks, ranks[1:], flats, flats[1:]):
            if p != q and a - b <= 2 * TOL:
                return False
    return True


CASES = [(1, 1, 1, 1, F32), (1, 1, 2, 4, F32), (2, 3, 10, 3, BF16), (1, 4, 50257, 4, BF16), (3, 4, 50257, 8, BF16),
         (2, 16, 1001, 16, F32), (1, 1, 50257, 5, F32), (5, 7, 2048, 7, BF16), (4, 2, 1025, 1, F32), (1, 64, 300, 64, F32),
         (1, 3, 7, 64, BF16), (1, 2, 262145, 12, BF16), (1, 2, 200003, 64, F32), (2, 33, 4097, 40, BF16)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "%d-%d-%d-%d-%s" % (*c[:4], str(c[4])[6:]))
@pytest.mark.parametrize("penalty", [0.0, 0.7])
def test_choices(case, penalty):
    require_gpu()
    R, W, V, K, dtype = case
    x, scores, done, lengths = draw(R, W, V, dtype, seed=R + W + V + K)
    eos = V // 2
    got = libks.beam_select(x, scores, K, done, lengths, eos, penalty)
    check(x, scores, K, done, lengths, eos, penalty, got, gaps(x, scores, done, lengths, eos, penalty, K))
    again = libks.beam_select(x, scores, K, done, lengths, eos, penalty)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_without_eos_and_lengths():
    require_gpu()
    x, scores, done, lengths = draw(3, 4, 999, F32, seed=2)
    got = libks.beam_select(x, scores)
    assert got.done is None and got.lengths is None
    check(x, scores, 4, None, None, None, 0.0, got)
    got = libks.beam_select(x, scores, 2, eos=5)              # none has ended so far
    check(x, scores, 2, None, None, 5, 0.0, got)
    got = libks.beam_select(x, scores, 6, lengths=lengths, length_penalty=1.5)
    check(x, scores, 6, None, lengths, None, 1.5, got)


def test_equal_candidates_go_by_beam_and_token():
    require_gpu()
    for dtype, V in ((F32, 5), (BF16, 2500), (F32, 5000)):
        # the same row in every beam, and few values in it
        row = torch.randint(0, 3, (V,), generator=torch.Generator().manual_seed(V)).to(dtype)
        x = row.expand(2, 4, V).contiguous().to(DEV)
        scores = torch.full((2, 4), -1.5, device=DEV)
        got = libks.beam_select(x, scores, 9)
        highest = (row == row.max()).nonzero()[:, 0]
        flat = [(w, int(t)) for w in range(4) for t in highest][:9]
        for r in range(2):
            assert list(zip(got.parents[r].tolist(), got.tokens[r].tolist()))[:len(flat)] == flat
        x.zero_()                                             # all of them
        x[0, :, ::2] = -0.0                                   # -0 is 0
        got = libks.beam_select(x, scores, 7)
        flat = [(w, t) for w in range(4) for t in range(V)][:7]
        for r in range(2):
            assert list(zip(got.parents[r].tolist(), got.tokens[r].tolist())) == flat


def test_sorted_and_constant_rows_fill_the_lists():
    """Values in an order that puts the best of them all in a few lanes."""
    require_gpu()
    V = 9000
    up = torch.arange(V, dtype=torch.float32) / 1000
    rows = torch.stack([up, up.flip(0), torch.full((V,), 2.0), (up * 7).floor()])
    x = rows[:, None, :].expand(4, 2, V).contiguous().to(DEV)
    scores = torch.tensor([[0.0, -0.25]]).expand(4, 2).contiguous().to(DEV)
    for K in (1, 5, 32, 64):
        check(x, scores, K, None, None, None, 0.0, libks.beam_select(x, scores, K),
              gaps(x, scores, None, None, None, 0.0, K))


def test_scores_a_step_apart():
    """Ranks that differ in the last bits of an fp32 score alone; two are equal."""
    require_gpu()
    V = 3000
    x = (-torch.arange(V, dtype=torch.float32)).expand(1, 4, V).contiguous().to(DEV)
    s = torch.tensor([-1.0])
    up, down = torch.nextafter(s, s + 1), torch.nextafter(s, s - 1)
    for order in ([s, down, up, s], [down, s, s, up], [up, up, down, s], [down, down, down, down]):
        scores = torch.cat(order)[None].to(DEV)
        want = sorted(range(4), key=lambda w: (-float(order[w]), w))
        got = libks.beam_select(x, scores, 8)
        assert got.parents[0].tolist() == want + want
        assert got.tokens[0].tolist() == [0] * 4 + [1] * 4
        assert bool((got.scores[0, :-1] >= got.scores[0, 1:]).all())


def test_beams_that_ended():
    require_gpu()
    x, scores, done, lengths = draw(6, 5, 700, BF16, seed=5)
    done[0] = True                                            # all of a request
    done[1] = False
    done[2, 1:] = True
    x[done] = float("nan")                                    # their logits are not read
    got = libks.beam_select(x, scores, 5, done, lengths, 3, 0.5)
    check(x, scores, 5, done, lengths, 3, 0.5, got)
    assert sorted(got.parents[0].tolist()) == [0, 1, 2, 3, 4] and got.done[0].all()


def test_banned_tokens_and_rows_that_cannot_be():
    require_gpu()
    for dtype in (F32, BF16):
        x, scores, _, _ = draw(8, 3, 400, dtype, seed=6)
        low = torch.finfo(dtype).min
        x[0, :, 4:] = float("-inf")                           # 12 candidates are left
        x[1, 0] = float("-inf")                               # a beam without any
        x[2] = float("-inf")                                  # a request without any
        x[3, :, 4:] = low                                     # the type's lowest value is a value
        x[4, 1, 7] = float("nan")
        x[5, 2, 9] = float("inf")
        scores[6, 1:] = float("-inf")                         # the first step: one beam
        scores[7, 0], scores[7, 1] = float("nan"), float("inf")
        got = libks.beam_select(x, scores, 16)
        keep = [0, 1, 2, 4, 5, 6, 7]
        check(x[keep], scores[keep], 16, None, None, None, 0.0, libks.Beams(*(None if t is None else t[keep] for t in got)))
        b = libks.beam_select(x[3:4], scores[3:4], 12)
        check(x[3:4], scores[3:4], 12, None, None, None, 0.0, b)
        assert bool((got.tokens[3, :12] < 4).all())
        # what nothing continues is done, and stays out of the next step
        b = libks.beam_select(x[2:3], scores[2:3], 3, eos=1)
        assert b.done.all() and bool((b.scores == -math.inf).all()) and b.tokens.tolist() == [[1, 1, 1]]
        b = libks.beam_select(x[6:7], b.scores, 3, b.done, eos=1)
        assert b.done.all() and bool((b.scores == -math.inf).all())


def test_strides():
    require_gpu()
    big, scores, _, _ = draw(3, 4, 1030, BF16, seed=7)
    for off in (0, 1, 3, 8):
        x = big[:, :, off:off + 1001]
        check(x, scores, 4, None, None, None, 0.0, libks.beam_select(x, scores))
    x = torch.randn(3, 9, 4, 500, device=DEV)[:, -1]          # the last position of a forward pass
    check(x, scores, 4, None, None, None, 0.0, libks.beam_select(x, scores))


@pytest.mark.parametrize("shape", [(1, 1, 1), (3, 4, 7), (2, 5, 1024), (2, 3, 40000)], ids=str)
@pytest.mark.parametrize("dtype", [torch.uint8, BF16, torch.int32, torch.float64], ids=lambda d: str(d)[6:])
def test_reorder(shape, dtype):
    require_gpu()
    R, W, n = shape
    g = torch.Generator().manual_seed(n)
    t = torch.randint(0, 200, (R, W, n), generator=g).to(dtype).to(DEV)
    u = torch.randint(0, 200, (R, W, 2, 3), generator=g).to(torch.int64).to(DEV)
    for beams in (1, W, 6):
        parents = torch.randint(W, (R, beams), generator=g, dtype=torch.int32).to(DEV)
        at = parents.long()
        rows = torch.arange(R, device=DEV)[:, None]
        got = libks.beam_reorder([t, u], parents)
        assert torch.equal(got[0], t[rows, at]) and torch.equal(got[1], u[rows, at])
        out = [torch.empty_like(v) for v in got]
        versions = [v._version for v in out]
        assert all(a is b for a, b in zip(libks.beam_reorder([t, u], parents, out=out), out))
        assert torch.equal(out[0], got[0]) and torch.equal(out[1], got[1])
        assert all(v._version > old for v, old in zip(out, versions))


def test_reorder_of_many_states_and_odd_places():
    require_gpu()
    g = torch.Generator().manual_seed(3)
    states = [torch.randint(0, 250, (2, 3, n), generator=g).to(torch.uint8).to(DEV) for n in range(1, 150)]
    buf = torch.randint(0, 250, (6 * 64 + 16,), generator=g).to(torch.uint8).to(DEV)
    states += [buf[off:off + 6 * 64].view(2, 3, 64) for off in (1, 4, 8)]
    parents = torch.tensor([[2, 2, 0], [1, 0, 7]], dtype=torch.int32, device=DEV)
    got = libks.beam_reorder(states, parents)
    for s, t in zip(states, got):
        assert torch.equal(t[0], s[0][[2, 2, 0]]) and torch.equal(t[1, :2], s[1][[1, 0]])
        assert not t[1, 2].any()                              # a parent that is not there
    assert libks.beam_reorder([], parents) == []
    empty = torch.empty(2, 3, 0, device=DEV)
    assert libks.beam_reorder([empty], parents)[0].shape == (2, 3, 0)


def test_reorder_past_4_gib():
    require_gpu()
    t = torch.zeros(3, 2, 1 << 30, dtype=torch.uint8, device=DEV)
    t[:, 0, -1], t[:, 1, -1], t[2, 1, 5] = 1, 2, 9
    parents = torch.tensor([[1, 0], [1, 1], [0, 1]], dtype=torch.int32, device=DEV)
    got, = libks.beam_reorder([t], parents)
    assert got[:, :, -1].tolist() == [[2, 1], [2, 2], [1, 2]] and got[2, :, 5].tolist() == [0, 9]
    assert int(got[2, 1, :1 << 20].sum()) == 9


def test_logits_past_2_31_elements():
    require_gpu()
    R, W, V = 700, 64, 50_257
    x = torch.zeros(R, W, V, dtype=BF16, device=DEV)
    x[-1].normal_(generator=torch.Generator(device=DEV).manual_seed(1))
    x[-1] *= 3
    scores = torch.zeros(R, W, device=DEV)
    scores[-1] = torch.linspace(-1, 0, W)
    got = libks.beam_select(x, scores, 4)
    check(x[-1:], scores[-1:], 4, None, None, None, 0.0, libks.Beams(*(None if t is None else t[-1:] for t in got)))
    assert got.tokens[:-1].tolist() == [[0, 1, 2, 3]] * (R - 1) and not got.parents[:-1].any()


def test_a_search_finds_what_enumeration_finds():
    """Select and reorder over several steps, with all continuations kept: the beams
    are the best of all sequences."""
    require_gpu()
    g = torch.Generator().manual_seed(11)
    V, steps, W = 4, 3, 64
    table = torch.randn(steps, V + 1, V, generator=g)         # logits by the token before
    scores = torch.full((2, 1), 0.0, device=DEV)
    history = torch.full((2, 1, 1), V, dtype=torch.int64, device=DEV)
    for s in range(steps):
        x = table[s].to(DEV)[history[:, :, -1]]
        b = libks.beam_select(x, scores, W)
        history, = libks.beam_reorder([history], b.parents)
        history = torch.cat([history, b.tokens[:, :, None]], dim=2)
        scores = b.scores
    log = torch.log_softmax(table.double(), dim=2)
    every = [((i, j, k), float(log[0, V, i] + log[1, i, j] + log[2, j, k]))
             for i in range(V) for j in range(V) for k in range(V)]
    every.sort(key=lambda c: -c[1])
    assert min(a[1] - b[1] for a, b in zip(every, every[1:])) > 3 * TOL
    for r in range(2):
        assert [tuple(t[1:]) for t in history[r].tolist()] == [c[0] for c in every]
        assert max(abs(a - c[1]) for a, c in zip(scores[r].tolist(), every)) <= 3 * TOL + 1e-6


def test_graph_and_streams():
    require_gpu()
    x, scores, done, lengths = draw(5, 4, 3001, BF16, seed=9)
    state = torch.randn(5, 4, 333, device=DEV)
    side = torch.cuda.Stream()
    want = libks.beam_select(x, scores, 4, done, lengths, 2, 0.5)
    moved = libks.beam_reorder([state], want.parents)
    side.wait_stream(torch.cuda.current_stream())
    got = libks.beam_select(x, scores, 4, done, lengths, 2, 0.5, stream=side)
    again = libks.beam_reorder([state], got.parents, stream=side)
    side.synchronize()
    assert isinstance(got, libks.Beams) and all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(again[0], moved[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b = libks.beam_select(x, scores, 4, done, lengths, 2, 0.5)
        s, = libks.beam_reorder([state], b.parents)
    for _ in range(4):
        x.normal_()
        scores.normal_()
        want = libks.beam_select(x, scores, 4, done, lengths, 2, 0.5)
        s.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(b, want))
        assert torch.equal(s, libks.beam_reorder([state], want.parents)[0])


def test_no_requests():
    require_gpu()
    b = libks.beam_select(torch.empty(0, 3, 10, device=DEV), torch.empty(0, 3, device=DEV), 4, eos=1)
    assert b.scores.shape == b.tokens.shape == b.done.shape == (0, 4)
    assert libks.beam_reorder([torch.empty(0, 3, 5, device=DEV)], b.parents)[0].shape == (0, 4, 5)


def test_refusals():
    require_gpu()
    x, scores, done, lengths = draw(2, 3, 20, F32, seed=1)
    bad = [dict(scores=scores[:, :2]), dict(scores=scores.double()), dict(done=done), dict(done=done.int(), eos=1),
           dict(length_penalty=1.0), dict(eos=20), dict(eos=-1), dict(lengths=lengths.long()),
           dict(scores=scores.t().contiguous().t()), dict(logits=x[0]), dict(logits=x.half()),
           dict(logits=x.transpose(1, 2).contiguous().transpose(1, 2)), dict(scores=scores.cpu())]
    for kw in bad:
        with pytest.raises((ValueError, TypeError)):
            libks.beam_select(**{"logits": x, "scores": scores, **kw})
    for kw in (dict(beams=0), dict(beams=65), dict(lengths=lengths, length_penalty=-1.0)):
        with pytest.raises(libks.KSError):
            libks.beam_select(x, scores, **kw)
    p = torch.zeros(2, 3, dtype=torch.int32, device=DEV)
    for args in (([x], p.long()), ([x], p[:1]), ([x[:, :, ::2]], p), ([x, x[:, :2].contiguous()], p), ([x], p, [x[:1]]),
                 ([x], p, []), ([x], p.cpu()), ([scores[:, 0]], p)):
        with pytest.raises((ValueError, TypeError)):
            libks.beam_reorder(*args)
    with pytest.raises(libks.KSError):
        libks.beam_reorder([x], p, out=[x])
