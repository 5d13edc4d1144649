"""What the calls write into a caller's tensors counts as an in-place change
(needs an MI355X): autograd and handles that keep something made from a tensor
notice, as they do for torch's own operations."""
from __future__ import annotations

import pytest
import torch

from gpu_helpers import DEV, require_gpu
from kronecker_sparse_structured_amd import layer, libks, optim
from test_gpu_adapters import draw

pytestmark = pytest.mark.gpu

CHAIN = [(3, 5, 7, 2), (1, 4, 30, 1)]        # 42 -> 30 -> 4: no chain that reads W itself
BITS = [32, 8]


def chain_of(t=torch.float32, patterns=CHAIN):
    n_in = patterns[0][0] * patterns[0][2] * patterns[0][3]
    n_out = patterns[-1][0] * patterns[-1][1] * patterns[-1][3]
    X, A, B, scale, ids = draw(70, n_in, n_out, 3, 5, t, t, seed=1, mix="random")
    g = torch.Generator().manual_seed(2)
    Ws = [(torch.randn(a, d, b, c, generator=g) / c ** 0.5).to(t).to(DEV) for a, b, c, d in patterns]
    return X, A, B, scale, ids, Ws, torch.randn(70, n_out, device=DEV)


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
def test_transposed_blocks_after_a_step_of_this_optimizer(bits, t):
    require_gpu()
    X, A, B, scale, ids, Ws, dY = chain_of(t)
    ready = libks.AdapterChain(Ws, CHAIN, A, B, scale, transposed=True)
    _, H = ready.matmul(X, ids, keep=True)
    before = ready.backward(dY, X, H, ids)[0]
    params = [torch.nn.Parameter(w) for w in Ws]                  # the same memory and counter
    opt = optim.AdamW(params, lr=0.1, state_bits=bits)
    for p in params:
        p.grad = torch.ones_like(p)
    opt.step()
    got = ready.backward(dY, X, H, ids)[0]
    want = libks.AdapterChain(Ws, CHAIN, A, B, scale).backward(dY, X, H, ids)[0]
    assert torch.equal(got, want) and not torch.equal(got, before)


@pytest.mark.parametrize("bits", BITS)
def test_a_step_between_forward_and_backward_is_seen(bits):
    require_gpu()
    base = layer.KSLinear(CHAIN, device=DEV)
    m = layer.AdapterLinear(base, 3, 5)
    x = torch.randn(70, 42, device=DEV)
    ids = torch.zeros(70, dtype=torch.int32, device=DEV)
    opt = optim.AdamW(m.parameters(), lr=0.1, state_bits=bits)
    m(x, ids).sum().backward()
    y = m(x, ids)
    opt.step()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


@pytest.mark.parametrize("views", [False, True])
@pytest.mark.parametrize("bits", BITS)
def test_every_tensor_of_a_step_is_counted(bits, views):
    require_gpu()
    sizes = [256, 512, 100]

    def make(dtype):
        if not views:
            return [torch.zeros(n, dtype=dtype, device=DEV) for n in sizes]
        flat = torch.zeros(1024, dtype=dtype, device=DEV)
        return [flat[a:a + n] for a, n in zip((0, 256, 768), sizes)]

    ps, gs = make(torch.float32), make(torch.float32)
    ms, vs = (make(torch.float32), make(torch.float32)) if bits == 32 else (make(torch.int8), make(torch.uint8))
    scales = None if bits == 32 else [torch.zeros(-(-n // 256), 2, device=DEV) for n in sizes]
    opt = libks.AdamW(ps, gs, ms, vs, scales)
    written, kept = [*ps, *ms, *vs, *(scales or ())], gs
    before, was = [t._version for t in written], [t._version for t in kept]
    opt.step(1, lr=0.1)
    assert all(t._version > v for t, v in zip(written, before))
    assert [t._version for t in kept] == was


def test_every_given_output_is_counted():
    require_gpu()
    X, A, B, scale, ids, Ws, dY = chain_of()
    chain = libks.AdapterChain(Ws, CHAIN, A, B, scale)
    _, H = chain.matmul(X, ids, keep=True)
    f32 = dict(dtype=torch.float32, device=DEV)
    logits = torch.randn(2, 3, 9, **f32)
    labels = torch.zeros(2, 3, dtype=torch.int64, device=DEV)
    p, m, v = (torch.zeros(300, dtype=t, device=DEV) for t in (torch.float32, torch.int8, torch.uint8))
    opt = libks.AdamW([p], [torch.ones(300, **f32)], [m], [v], [torch.zeros(2, 2, **f32)])
    one = CHAIN[0]
    calls = [
        (torch.empty(70, 4, **f32), lambda t: chain.matmul(X, ids, out=t)),
        (torch.zeros(70, 4, **f32), lambda t: libks.adapter_matmul(X, A, B, scale, ids, t)),
        (torch.zeros(70, 42, **f32), lambda t: libks.adapter_backward(dY, X, H, A, B, scale, ids, dX=t)),
        (torch.empty(70, 30, **f32), lambda t: libks.matmul(X, Ws[0], one, out=t)),
        (torch.empty(70, 4, **f32), lambda t: libks.chain_matmul(X, Ws, CHAIN, out=t)),
        (torch.empty(70, 42, **f32), lambda t: libks.matmul_dx(torch.ones(70, 30, **f32), Ws[0], one, out=t)),
        (torch.empty_like(Ws[0]), lambda t: libks.matmul_dw(torch.ones(70, 30, **f32), X, one, out=t)),
        (logits, lambda t: libks.preference_loss(t, labels, torch.zeros(2, 3, **f32), dlogits=t)),
        (torch.empty((), **f32), lambda t: opt.grad_norm(out=t)),
        (torch.empty(300, **f32), lambda t: opt.state_values([t], [torch.empty(300, **f32)])),
        (torch.empty(300, **f32), lambda t: opt.state_values([torch.empty(300, **f32)], [t])),
    ]
    for k, (t, call) in enumerate(calls):
        before = t._version
        call(t)
        assert t._version > before, k


def test_inference_tensors_have_no_counter():
    require_gpu()
    with torch.inference_mode():
        X, A, B, scale, ids, Ws, dY = chain_of()
        out = torch.empty(70, 4, device=DEV)
        libks.AdapterChain(Ws, CHAIN, A, B, scale).matmul(X, ids, out=out)
        p, g, m, v = (torch.ones(300, device=DEV) for _ in range(4))
        libks.AdamW([p], [g], [m], [v]).step(1, lr=0.1)
        assert float(p[0]) < 1.0


@pytest.mark.parametrize("what", ["W", "scale"])
def test_a_change_of_what_is_frozen_between_forward_and_backward_is_seen(what):
    """dX is formed from W, E and dX from scale, H before: all of one time."""
    require_gpu()
    base = layer.KSLinear(CHAIN, device=DEV)
    m = layer.AdapterLinear(base, 3, 5)
    x = torch.randn(70, 42, device=DEV, requires_grad=True)
    ids = torch.zeros(70, dtype=torch.int32, device=DEV)
    y = m(x, ids)
    with torch.no_grad():
        (base.weights[1] if what == "W" else m.scale).mul_(2)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    m(x, ids).sum().backward()
    assert x.grad.any()


def test_frozen_weights_that_are_inference_tensors_train_adapters():
    require_gpu()
    with torch.inference_mode():
        base = layer.KSLinear(CHAIN, device=DEV)
        for w in base.weights:
            w.requires_grad_(False)
    m = layer.AdapterLinear(base, 3, 5)
    m.A, m.B, m.scale = (torch.nn.Parameter(torch.ones_like(m.A)), torch.nn.Parameter(torch.ones_like(m.B)),
                         torch.ones(3, device=DEV))
    x = torch.randn(70, 42, device=DEV)
    m(x, torch.zeros(70, dtype=torch.int32, device=DEV)).sum().backward()
    assert m.A.grad[0].any() and m.B.grad[0].any()


def test_transposed_blocks_of_inference_tensors():
    require_gpu()
    with torch.inference_mode():
        X, A, B, scale, ids, Ws, dY = chain_of()
        ready = libks.AdapterChain(Ws, CHAIN, A, B, scale, transposed=True)
        plain = libks.AdapterChain(Ws, CHAIN, A, B, scale)
        _, H = ready.matmul(X, ids, keep=True)
        for _ in range(2):
            assert all(torch.equal(a, b) for a, b in zip(ready.backward(dY, X, H, ids), plain.backward(dY, X, H, ids)))
            Ws[0].mul_(2)
    X, A, B, scale, ids, Ws, dY = chain_of()
    with torch.inference_mode():                 # tensors made outside keep their version
        ready = libks.AdapterChain(Ws, CHAIN, A, B, scale, transposed=True)
        assert ready._wt is not None
        _, H = ready.matmul(X, ids, keep=True)
        before = ready.backward(dY, X, H, ids)[0]
        Ws[0].mul_(2)
        assert torch.equal(ready.backward(dY, X, H, ids)[0],
                           libks.AdapterChain(Ws, CHAIN, A, B, scale).backward(dY, X, H, ids)[0])
        assert not torch.equal(ready.backward(dY, X, H, ids)[0], before)
