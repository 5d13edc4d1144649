"""Calls with a ``stream`` of their own (needs an MI355X): results are those of
the call on torch's current stream, and nothing that the kernels there still use
is handed to another stream's allocations when the call returns."""
from __future__ import annotations

import pytest
import torch

from gpu_helpers import DEV, require_gpu
from kronecker_sparse_structured_amd import libks
from test_gpu_adapters import BF16, F32, PAIR, draw

pytestmark = pytest.mark.gpu


class Recorder:
    """libks with the pointer arguments of every call noted."""

    def __init__(self, lib):
        self.lib, self.seen, self.streams = lib, set(), set()

    def __getattr__(self, name):
        fn = getattr(self.lib, name)

        def call(*args):
            self.seen |= {a for a in args if isinstance(a, int) and a > 1 << 32}
            if not name.endswith("_size"):
                self.streams.add(args[-2] if name == "ks_matmul_ex" else args[-1])
            return fn(*args)

        return call


def flat(x):
    return [t for y in (x if isinstance(x, tuple) else (x,)) for t in ([y] if isinstance(y, torch.Tensor) else [])]


def problems():
    """name: (inputs, call(stream, inputs)) with fresh results or changed copies returned."""
    out = {}
    g = torch.Generator(device=DEV).manual_seed(3)
    ps = [(2, 8, 8, 4), (4, 4, 4, 4), (1, 16, 64, 1), (4, 3, 4, 1)]
    Ws = [torch.randn(a, d, b, c, device=DEV, generator=g) for a, b, c, d in ps]
    X = torch.randn(3000, 64, device=DEV, generator=g)
    dZ = torch.randn(3000, 64, device=DEV, generator=g)
    out["matmul"] = lambda s: libks.matmul(X, Ws[0], ps[0], stream=s)
    out["chain_matmul"] = lambda s: libks.chain_matmul(X, Ws, ps, fuse=False, stream=s)
    out["matmul_dx"] = lambda s: libks.matmul_dx(dZ, Ws[0], ps[0], stream=s)
    out["matmul_dw"] = lambda s: libks.matmul_dw(dZ, X, ps[0], stream=s)
    for batch, t in ((40, F32), (1500, BF16)):
        x, A, B, scale, ids = draw(batch, 1024, 4096, 3, 16, t, t, seed=batch)
        W = [(torch.randn(a, d, b, c, generator=g, device=DEV) / c ** 0.5).to(t) for a, b, c, d in PAIR]
        dY = torch.randn(batch, 4096, device=DEV, generator=g)
        chain = libks.AdapterChain(W, PAIR, A, B, scale, transposed=t == F32)
        H = chain.matmul(x, ids, keep=True)[1]
        key = "_%d" % batch
        out["chain" + key] = lambda s, c=chain, x=x, i=ids: c.matmul(x, i, stream=s)
        out["chain_keep" + key] = lambda s, c=chain, x=x, i=ids: c.matmul(x, i, keep=True, stream=s)
        out["chain_backward" + key] = lambda s, c=chain, x=x, i=ids, y=dY, h=H: c.backward(y, x, h, i, stream=s)

        def add(s, x=x, a=(A, B, scale, ids), y=dY):
            y = y.clone()
            torch.cuda.synchronize()
            return libks.adapter_matmul(x, *a, y, stream=s)

        out["adapter" + key] = add
        out["adapter_backward" + key] = \
            lambda s, x=x, h=H, a=(A, B, scale, ids), y=dY: libks.adapter_backward(y, x, h, *a, stream=s)
    logits = torch.randn(4, 70, 1000, device=DEV, generator=g)
    labels = torch.randint(1000, (4, 70), device=DEV, generator=g)
    ref = torch.randn(4, 70, device=DEV, generator=g) - 7
    out["sequence_logp"] = lambda s: libks.sequence_logp(logits, labels, stream=s)
    out["preference_loss"] = lambda s: libks.preference_loss(logits, labels, ref, stream=s)
    grads = [torch.randn(n, device=DEV, generator=g) for n in (5000, 70000, 3)]

    def step(s):
        p, m, v = ([torch.ones_like(t) for t in grads] for _ in range(3))
        torch.cuda.synchronize()
        opt = libks.AdamW(p, grads, m, v)
        out = opt.step(1, lr=0.1, max_norm=0.5, stream=s), opt.grad_norm(stream=s), *p, *m, *v
        return out

    out["adamw"] = step
    return out


NAMES = ["matmul", "chain_matmul", "matmul_dx", "matmul_dw", "chain_40", "chain_keep_40", "chain_backward_40", "adapter_40",
         "adapter_backward_40", "chain_1500", "chain_keep_1500", "chain_backward_1500", "adapter_1500",
         "adapter_backward_1500", "sequence_logp", "preference_loss", "adamw"]


@pytest.mark.parametrize("kind", ["object", "address"])
@pytest.mark.parametrize("name", NAMES)
def test_memory_of_a_call_on_another_stream(name, kind, monkeypatch):
    require_gpu()
    call = problems()[name]
    want = [t.clone() for t in flat(call(None))]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    rec = Recorder(libks.load())
    monkeypatch.setattr(libks, "_lib", rec)
    got = flat(call(side if kind == "object" else side.cuda_stream))
    monkeypatch.undo()
    if not rec.seen:                             # a handle keeps the library it was made with: the results alone
        rec.streams.add(side.cuda_stream)
    assert rec.streams == {side.cuda_stream}
    # what this stream gets from now on: none of what the call used
    mine = [torch.full((n,), 255, dtype=torch.uint8, device=DEV)
            for n in (256, 1024, 4096, 20000, 100000, 400000, 1 << 20, 3 << 20, 20 << 20) for _ in range(6)]
    for t in mine:
        a = t.data_ptr()
        assert not any(a <= p < a + t.numel() for p in rec.seen), name
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_handle_on_another_stream():
    """The handles note their library once: here with the recorder in place."""
    require_gpu()
    x, A, B, scale, ids = draw(1500, 1024, 4096, 3, 16, BF16, BF16, seed=1)
    W = [(torch.randn(a, d, b, c) / c ** 0.5).to(BF16).to(DEV) for a, b, c, d in PAIR]
    dY = torch.randn(1500, 4096, device=DEV)
    chain = libks.AdapterChain(W, PAIR, A, B, scale)
    want = *chain.matmul(x, ids, keep=True), *chain.backward(dY, x, chain.matmul(x, ids, keep=True)[1], ids)
    want = [t.clone() for t in want]
    chain._lib = rec = Recorder(libks.load())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    Y, H = chain.matmul(x, ids, keep=True, stream=side)
    got = [Y, H, *chain.backward(dY, x, H, ids, stream=side)]
    chain.matmul(x, ids, stream=side)            # H and its parts in the workspace
    assert rec.streams == {side.cuda_stream} and rec.seen
    mine = [torch.full((n,), 255, dtype=torch.uint8, device=DEV)
            for n in (256, 4096, 20000, 100000, 400000, 1 << 20, 3 << 20, 30 << 20) for _ in range(6)]
    for t in mine:
        assert not any(t.data_ptr() <= p < t.data_ptr() + t.numel() for p in rec.seen)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    opt = libks.AdamW([Y], [torch.ones_like(Y)], [torch.zeros_like(Y)], [torch.zeros_like(Y)])
    opt._lib = rec = Recorder(libks.load())
    torch.cuda.synchronize()
    norm = opt.step(1, lr=0.1, max_norm=1.0, stream=side)
    assert rec.streams == {side.cuda_stream}
    more = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in (256, 512, 4096, 65536, 1 << 20) for _ in range(6)]
    for t in more:
        assert not any(t.data_ptr() <= p < t.data_ptr() + t.numel() for p in rec.seen)
    side.synchronize()
    assert abs(float(norm) - (1500 * 4096) ** 0.5) <= 1e-3 * 2500


def test_the_default_stream_by_its_address():
    require_gpu()
    X = torch.randn(64, 42, device=DEV)
    W = torch.randn(3, 2, 5, 7, device=DEV)
    want = libks.matmul(X, W, (3, 5, 7, 2))
    assert torch.equal(libks.matmul(X, W, (3, 5, 7, 2), stream=0), want)
    with torch.cuda.stream(torch.cuda.Stream()):
        got = libks.matmul(X, W, (3, 5, 7, 2), stream=torch.cuda.default_stream())
    torch.cuda.synchronize()
    assert torch.equal(got, want)
