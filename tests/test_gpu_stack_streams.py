"""Residual norms, distillation and beam search on streams, in threads, in graphs
and in inference mode (needs an MI355X): results are those of a plain call, and
nothing that kernels still use is handed to another stream's allocations."""
from __future__ import annotations

import threading

import pytest
import torch

import test_gpu_distillation as dist
import test_gpu_residual_norm as norms
from gpu_helpers import DEV, require_gpu
from kronecker_sparse_structured_amd import layer, libks
from test_gpu_beam_search import draw as draw_beams
from test_gpu_streams import Recorder

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def flat(x):
    if isinstance(x, torch.Tensor):
        return [x]
    return [t for y in x for t in flat(y)] if isinstance(x, (tuple, list)) else []


def problems():
    """name: call(stream) with fresh results."""
    out = {}
    for name, (S, T, V, K, t) in {"distil": (2, 40, 5000, 20, BF16), "distil_many": (3, 700, 90, 4, F32),
                                  "distil_long": (1, 3, 70001, 9, F32)}.items():
        data = dist.draw(S, T, V, K, t, seed=V)
        out[name] = lambda s, d=data: libks.distillation_loss(*d, 0.5, 2.0, stream=s)
        out[name + "_loss"] = lambda s, d=data: libks.distillation_loss(*d, 0.5, 2.0, grad=False, stream=s)[:2]
    x, scores, done, lengths = draw_beams(20, 5, 9001, BF16, seed=2)
    out["select"] = lambda s: libks.beam_select(x, scores, 5, done, lengths, 4, 0.5, stream=s)
    out["select_more"] = lambda s: libks.beam_select(x, scores, 9, stream=s)
    states = [torch.randn(20, 5, n, device=DEV) for n in (3, 1000, 40000)]
    parents = torch.randint(5, (20, 7), device=DEV, dtype=torch.int32)
    out["reorder"] = lambda s: libks.beam_reorder(states, parents, stream=s)
    p = norms.make(3000, 520, "layer", groups=6, x=BF16, seed=1)

    def norm(s):
        n = norms.handle(p)                      # made with the library of the moment
        z, h, stats = n.forward(p["x"], p["y"], p["gate"], dtype=BF16, keep=True, stream=s)
        dh = torch.ones_like(h) if s is None else p["dh16"]
        return z, h, stats, *n.backward(p["dz"], dh, p["x"], p["y"], stats, p["gate"], stream=s)

    p["dh16"] = torch.ones(3000, 520, dtype=BF16, device=DEV)
    out["norm"] = norm
    return out


NAMES = ["distil", "distil_loss", "distil_many", "distil_many_loss", "distil_long", "distil_long_loss", "select",
         "select_more", "reorder", "norm"]


@pytest.mark.parametrize("name", NAMES)
def test_memory_of_a_call_on_another_stream(name, monkeypatch):
    require_gpu()
    call = problems()[name]
    want = [t.clone() for t in flat(call(None))]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    rec = Recorder(libks.load())
    monkeypatch.setattr(libks, "_lib", rec)
    got = flat(call(side))
    monkeypatch.undo()
    assert rec.streams == {side.cuda_stream}
    mine = [torch.full((n,), 255, dtype=torch.uint8, device=DEV)
            for n in (256, 1024, 4096, 20000, 100000, 400000, 1 << 20, 3 << 20, 20 << 20) for _ in range(6)]
    for t in mine:
        a = t.data_ptr()
        assert not any(a <= p < a + t.numel() for p in rec.seen), name
    side.synchronize()
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_one_handle_from_two_threads():
    """Calls of different types on one handle at once: each has its own arguments."""
    require_gpu()
    p = norms.make(400, 384, "rms", groups=4, seed=3)
    n = norms.handle(p)
    kinds = [(F32, F32, F32), (BF16, F32, BF16), (F32, BF16, BF16), (BF16, BF16, F32)]
    inputs = [(p["x"].to(a), p["y"].to(b), c) for a, b, c in kinds]

    def work(x, y, c):
        z, h, stats = n.forward(x, y, p["gate"], dtype=c, keep=True)
        return z, h, *n.backward(p["dz"].to(x.dtype), p["dh"].to(c), x, y, stats, p["gate"])[:3]

    want = [[t.clone() for t in work(*i)] for i in inputs]
    torch.cuda.synchronize()
    bad = []

    def run(k):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(60):
                got = work(*inputs[k])
                stream.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[k])):
                    bad.append(k)

    threads = [threading.Thread(target=run, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_two_graphs_in_turn():
    require_gpu()
    graphs = []
    for seed in (1, 2):
        data = dist.draw(2, 30, 600, 8, BF16, seed=seed)
        x, scores, done, lengths = draw_beams(6, 4, 5001, F32, seed=seed)
        p = norms.make(900, 264, "layer", groups=3, seed=seed)
        n = norms.handle(p)

        def step(data=data, x=x, scores=scores, done=done, lengths=lengths, p=p, n=n):
            z, h, stats = n.forward(p["x"], p["y"], p["gate"], keep=True)
            return (libks.distillation_loss(*data, 0.5, 2.0), libks.beam_select(x, scores, 4, done, lengths, 1, 0.3),
                    z, h, n.backward(p["dz"], p["dh"], p["x"], p["y"], stats, p["gate"]))

        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out, step, (data[0], x, p["y"])))
    for turn in range(4):
        for g, out, step, inputs in graphs:
            for t in inputs:
                t.normal_()
        want = [[t.clone() for t in flat(step())] for _, _, step, _ in graphs]
        for g, out, _, _ in graphs if turn % 2 else graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        for (g, out, _, _), w in zip(graphs, want):
            assert all(torch.equal(a, b) for a, b in zip(flat(out), w)), turn


def test_calls_at_once_on_two_streams():
    require_gpu()
    calls = problems()
    names = ["distil", "select", "norm", "distil_many"]
    want = {k: [t.clone() for t in flat(calls[k](None))] for k in names}
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for s in streams:
            got += [(k, flat(calls[k](s))) for k in names]
        torch.cuda.synchronize()
        for k, ts in got:
            assert all(torch.equal(a, b) for a, b in zip(ts, want[k])), k


def test_given_gradients_count_as_changes():
    require_gpu()
    data = dist.draw(1, 4, 50, 6, F32, seed=1)
    x = data[0].clone().requires_grad_(True)
    y = x * 1.0
    z = (y * y).sum()                              # y is saved
    libks.distillation_loss(y.detach(), *data[1:], dlogits=y.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.backward()
    logits = data[0].clone().requires_grad_(True)
    loss, _ = layer.distillation_loss(logits, *data[1:])
    with torch.no_grad():
        logits.mul_(2)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_inference_mode():
    require_gpu()
    stack = layer.ResidualStack([layer.KSLinear([(4, 8, 8, 2)], device=DEV)], 64, post=True, scale=0.5, device=DEV)
    x = torch.randn(5, 64, device=DEV)
    with torch.no_grad():
        want = stack(x)
    with torch.inference_mode():
        got = stack(x.clone())
        assert torch.equal(got, want)
        logits = torch.randn(2, 3, 40, device=DEV)
        b = libks.beam_select(logits, torch.zeros(2, 3, device=DEV))
        state = torch.randn(2, 3, 4, device=DEV)
        out = torch.empty_like(state)
        libks.beam_reorder([state], b.parents, out=[out])
        assert torch.equal(out, state[torch.arange(2, device=DEV)[:, None], b.parents.long()])


def test_broadcast_gates_and_inputs_have_their_gradients():
    """An expanded gate or input: the gradient is summed over what it was expanded to."""
    require_gpu()
    m = layer.ResidualNorm(24, post=True, scale=0.5, device=DEV)
    g = torch.Generator().manual_seed(1)
    x, gate = torch.randn(1, 24, generator=g).to(DEV), (1 + torch.randn(24, generator=g)).to(DEV)
    y = torch.randn(6, 24, generator=g).to(DEV)
    got = []
    for spread in (False, True):
        a, b = x.clone().requires_grad_(True), gate.clone().requires_grad_(True)
        xs = a.expand(6, 24)
        if spread:
            xs = xs.contiguous()
        z, h = m(xs, y, b.expand(6, 24).contiguous() if spread else b.expand(1, 24))
        (z.square().sum() + h.sum()).backward()
        got.append((a.grad, b.grad))
    for s, t in zip(*got):
        # 6 rows' terms in another order, each off by the norm's N u times a few
        assert float((s - t).abs().max()) <= 1e-4 * float(t.abs().max())


def test_empty_batches_of_modules():
    require_gpu()
    m = layer.ResidualNorm(16, kind="layer", post=True, scale=1.0, device=DEV)
    x, y = (torch.empty(0, 4, 16, device=DEV, requires_grad=True) for _ in range(2))
    z, h = m(x, y)
    assert z.shape == h.shape == (0, 4, 16)
    (z.sum() + h.sum()).backward()
    assert x.grad.shape == (0, 4, 16) and not m.pre_weight.grad.any() and not m.scale.grad.any()
    logits = torch.empty(0, 3, 9, device=DEV, requires_grad=True)
    loss, _ = layer.distillation_loss(logits, torch.empty(0, 3, dtype=torch.int64, device=DEV),
                                      torch.empty(0, 3, 2, dtype=torch.int64, device=DEV),
                                      torch.empty(0, 3, 2, device=DEV))
    loss.backward()
    assert float(loss.detach()) == 0.0 and logits.grad.shape == (0, 3, 9)
