"""Adapters beside a KS projection (needs an MI355X) against the formula in
64 bits.

Tolerances. An fp32 sum of k terms is off by at most k 2^-24 sum |terms|, so a
product of two such sums (lengths k1, then k2) is off by at most about
(k1 + k2 + 2) 2^-24 of the same expression on magnitudes; twice that is allowed
(2^-23), which also covers the rounding of each product.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import DEV, FP32_REL_TOL, require_gpu
from kronecker_sparse_structured_amd import layer, libks

pytestmark = pytest.mark.gpu
U = 2.0 ** -23
F32, BF16 = torch.float32, torch.bfloat16


def draw(batch, n_in, n_out, count, rank, xt=F32, wt=F32, seed=0, mix="runs"):
    g = torch.Generator().manual_seed(seed)
    X = torch.randn(batch, n_in, generator=g).to(xt).to(DEV)
    A = (torch.randn(count, rank, n_in, generator=g) / n_in ** 0.5).to(wt).to(DEV)
    B = (torch.randn(count, n_out, rank, generator=g) / rank ** 0.5).to(wt).to(DEV)
    scale = (0.5 + torch.rand(count, generator=g)).to(DEV)
    ids = torch.randint(-1, count + 1, (batch,), generator=g)   # some outside on both sides
    if mix == "runs":
        ids = ids.sort().values.roll(batch // 3)
    elif mix == "one":
        ids[:] = count - 1
    elif mix == "none":
        ids[:] = -1
    return X, A, B, scale, ids.to(torch.int32).to(DEV)


def f64(*ts):
    return [t.detach().double().cpu() for t in ts]


def formula(X, A, B, scale, ids, dY=None):
    """H, delta (and E, dX, dA, dB) in 64 bits."""
    X, A, B, scale = f64(X, A, B, scale)
    ids = ids.cpu().long()
    on = (ids >= 0) & (ids < A.shape[0])
    g = ids.clamp(0, A.shape[0] - 1)
    H = torch.zeros(X.shape[0], A.shape[1], dtype=torch.float64)
    D = torch.zeros(X.shape[0], B.shape[1], dtype=torch.float64)
    out = {}
    E = torch.zeros_like(H)
    dX, dA, dB = torch.zeros_like(X), torch.zeros_like(A), torch.zeros_like(B)
    for a in range(A.shape[0]):
        r = (on & (g == a)).nonzero()[:, 0]
        H[r] = scale[a] * X[r] @ A[a].T
        D[r] = H[r] @ B[a].T
        if dY is not None:
            y = dY.double().cpu()[r]
            E[r] = scale[a] * y @ B[a]
            dX[r] = E[r] @ A[a]
            dA[a] = E[r].T @ X[r]
            dB[a] = y.T @ H[r]
    out.update(H=H, D=D, E=E, dX=dX, dA=dA, dB=dB)
    return out


def near(got, ref, mag, terms, what):
    err = (got.double().cpu() - ref).abs()
    bound = terms * U * mag + 1e-30
    assert bool((err <= bound).all()), "%s: worst ratio %g" % (what, float((err / bound).max()))


CASES = [
    # batch, n_in, n_out, count, rank, types, mix
    (1, 1024, 4096, 8, 16, (BF16, BF16), "one"), (1, 42, 30, 1, 5, (F32, F32), "one"),
    (2, 1, 1, 2, 1, (F32, F32), "random"), (5, 64, 20, 3, 4, (F32, BF16), "random"),
    (33, 40, 36, 7, 13, (BF16, BF16), "random"), (64, 384, 1536, 32, 8, (F32, F32), "random"),
    (200, 256, 384, 4, 256, (BF16, BF16), "runs"), (1024, 96, 160, 5, 17, (F32, F32), "random"),
    (1025, 96, 160, 5, 17, (F32, F32), "random"), (1030, 1024, 512, 9, 16, (BF16, BF16), "runs"),
    (1100, 42, 30, 3, 5, (BF16, BF16), "random"), (1500, 100, 68, 40, 24, (F32, BF16), "random"),
    (2049, 384, 1536, 2, 8, (F32, F32), "runs"), (3000, 1024, 256, 4, 33, (BF16, BF16), "runs"),
    (1040, 64, 64, 3, 200, (F32, F32), "random"), (1100, 128, 64, 3, 16, (F32, F32), "none"),
    (4099, 64, 1000, 2, 32, (BF16, BF16), "one"),
    # both sides of the gradients' limit of rows for two small launches
    (64, 300, 520, 1, 16, (BF16, BF16), "one"), (65, 300, 520, 3, 16, (BF16, BF16), "random"),
    (4, 260, 1, 2, 256, (F32, F32), "random"), (12, 1, 300, 5, 67, (F32, BF16), "random"),
    (9, 512, 96, 3, 100, (BF16, BF16), "none"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c[:5]) + "-" + c[6])
def test_forward_and_gradients(case):
    require_gpu()
    batch, n_in, n_out, count, rank, (xt, wt), mix = case
    X, A, B, scale, ids = draw(batch, n_in, n_out, count, rank, xt, wt, seed=batch + rank, mix=mix)
    Y0 = torch.randn(batch, n_out, device=DEV)
    dY = torch.randn(batch, n_out, device=DEV)
    dX0 = torch.randn(batch, n_in, device=DEV)
    ref = formula(X, A, B, scale, ids, dY)
    mag = formula(X.abs(), A.abs(), B.abs(), scale, ids, dY.abs())
    out = Y0.clone()
    Y, H = libks.adapter_matmul(X, A, B, scale, ids, out, keep=True)
    assert Y is out
    near(H, ref["H"], mag["H"], n_in + 2, "H")
    near(Y, Y0.double().cpu() + ref["D"], Y0.double().cpu().abs() + mag["D"], n_in + rank + 4, "Y")
    dX = dX0.clone()
    dA, dB = libks.adapter_backward(dY, X, H, A, B, scale, ids, dX=dX)
    near(dX, dX0.double().cpu() + ref["dX"], dX0.double().cpu().abs() + mag["dX"], n_out + rank + 4, "dX")
    near(dA, ref["dA"], mag["dA"], n_out + batch + 4, "dA")
    near(dB, ref["dB"], mag["dB"], n_in + batch + 4, "dB")
    # the same call again: identical bits
    dX2 = dX0.clone()
    dA2, dB2 = libks.adapter_backward(dY, X, H, A, B, scale, ids, dX=dX2)
    assert torch.equal(dA, dA2) and torch.equal(dB, dB2) and torch.equal(dX, dX2)
    # rows without an adapter keep their bits
    off = ((ids < 0) | (ids >= count))
    assert torch.equal(Y[off], Y0[off]) and torch.equal(dX[off], dX0[off]) and not H[off].any()


def test_gradients_against_differences():
    """The loss sum(Y * C) is linear in A and in B and quadratic along both: its
    central difference along a direction is exact up to rounding, in 64 bits."""
    require_gpu()
    X, A, B, scale, ids = draw(1500, 60, 52, 3, 6, seed=4, mix="random")
    C = torch.randn(1500, 52, device=DEV)
    H = torch.empty(1500, 6, device=DEV)
    _, H = libks.adapter_matmul(X, A, B, scale, ids, torch.zeros(1500, 52, device=DEV), keep=True)
    dX = torch.zeros_like(X)
    dA, dB = libks.adapter_backward(C, X, H, A, B, scale, ids, dX=dX)
    c = C.double().cpu()
    for name, base, grad in (("A", A, dA), ("B", B, dB), ("X", X, dX)):
        D = torch.randn(base.shape, generator=torch.Generator().manual_seed(9)).to(DEV)
        vals = []
        for sign in (1, -1):
            t = dict(X=X.double(), A=A.double(), B=B.double())
            t[name] = t[name] + sign * 1e-3 * D.double()
            vals.append(float((formula(t["X"], t["A"], t["B"], scale, ids)["D"] * c).sum()))
        num = (vals[0] - vals[1]) / 2e-3
        ana = float((grad.double().cpu() * D.double().cpu()).sum())
        # each gradient value is off by at most (52 + 1500) 2^-23 of its magnitude
        bound = 1552 * U * float((grad.double().cpu().abs() * D.double().cpu().abs()).sum()) * 4 + 1e-6
        assert abs(num - ana) <= bound, (name, num, ana)


def test_nan_and_infinity_stay_with_their_rows():
    require_gpu()
    for batch in (64, 1200):
        X, A, B, scale, ids = draw(batch, 64, 64, 4, 8, seed=batch, mix="random")
        A[1, 2, 3] = float("nan")
        B[2, 5] = float("inf")
        X[3] = float("nan")
        out = torch.zeros(batch, 64, device=DEV)
        Y, H = libks.adapter_matmul(X, A, B, scale, ids, out, keep=True)
        clean = (ids != 1) & (ids != 2)
        clean[3] = False
        assert torch.isfinite(Y[clean]).all() and torch.isfinite(H[clean]).all()
        off = (ids < 0) | (ids >= 4)
        assert not Y[off].any()
        assert not torch.isfinite(Y[ids == 1]).any(dim=1)[Y[ids == 1].abs().sum(1) == 0].any()
        dX = torch.zeros(batch, 64, device=DEV)
        dA, dB = libks.adapter_backward(torch.ones(batch, 64, device=DEV), X, H, A, B, scale, ids, dX=dX)
        own = [g for g in (0, 3) if not bool((ids[3] == g))]
        assert all(torch.isfinite(dA[g]).all() and torch.isfinite(dB[g]).all() for g in own)
        assert torch.isfinite(dX[clean]).all()


def test_adapters_without_rows_get_zero_gradients():
    require_gpu()
    X, A, B, scale, ids = draw(300, 32, 48, 6, 8, seed=1, mix="one")
    H = libks.adapter_matmul(X, A, B, scale, ids, torch.zeros(300, 48, device=DEV), keep=True)[1]
    dA, dB = libks.adapter_backward(torch.ones(300, 48, device=DEV), X, H, A, B, scale, ids)
    assert not dA[:5].any() and not dB[:5].any() and dA[5].any() and dB[5].any()
    empty = torch.empty(0, 32, device=DEV)
    dA, dB = libks.adapter_backward(torch.empty(0, 48, device=DEV), empty, torch.empty(0, 8, device=DEV), A, B, scale,
                                    torch.empty(0, dtype=torch.int32, device=DEV))
    assert not dA.any() and not dB.any()


def test_unaligned_pointers():
    require_gpu()
    for batch in (40, 1300):
        X, A, B, scale, ids = draw(batch, 64, 32, 3, 8, seed=2, mix="runs")
        dY = torch.randn(batch, 32, device=DEV)

        def shifted(t):
            flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
            flat[1:] = t.reshape(-1)
            return flat[1:].view(t.shape)

        a = [torch.zeros(batch, 32, device=DEV), torch.zeros(batch, 64, device=DEV)]
        b = [shifted(t) for t in a]
        H = libks.adapter_matmul(X, A, B, scale, ids, a[0], keep=True)[1]
        Hs = libks.adapter_matmul(shifted(X), shifted(A), shifted(B), scale, ids, b[0], keep=True)[1]
        g = libks.adapter_backward(dY, X, H, A, B, scale, ids, dX=a[1])
        gs = libks.adapter_backward(shifted(dY), shifted(X), shifted(Hs), shifted(A), shifted(B), scale, ids, dX=b[1])
        for x, y in zip((H, *a, *g), (Hs, *b, *gs)):
            assert torch.allclose(x, y, rtol=1e-4, atol=1e-4)


CHAINS = [([(1, 64, 16, 64), (64, 8, 8, 8)], 5, BF16), ([(1, 64, 16, 64), (64, 8, 8, 8)], 6007, BF16),
          ([(4, 64, 16, 6)], 1111, F32), ([(3, 5, 7, 2)], 77, F32), ([(3, 5, 7, 2)], 1500, BF16),
          ([(32, 32, 32, 1), (1, 32, 32, 32)], 1200, F32), ([(2 ** k, 2, 2, 2 ** (9 - k)) for k in range(10)], 300, F32)]


@pytest.mark.parametrize("case", CHAINS, ids=lambda c: "%dx%d" % (len(c[0]), c[1]))
def test_chain_with_adapters(case):
    require_gpu()
    ps, batch, t = case
    n_in, n_out = ps[0][0] * ps[0][2] * ps[0][3], ps[-1][0] * ps[-1][1] * ps[-1][3]
    X, A, B, scale, ids = draw(batch, n_in, n_out, 3, 8, t, t, seed=batch, mix="runs")
    Ws = [(torch.randn(a, d, b, c) / c ** 0.5).to(t).to(DEV) for a, b, c, d in ps]
    chain = libks.AdapterChain(Ws, ps, A, B, scale)
    Y, H = chain.matmul(X, ids, keep=True)
    assert torch.equal(Y, chain.matmul(X, ids))
    dY = torch.randn(batch, n_out, device=DEV)
    dX, dA, dB = chain.backward(dY, X, H, ids)
    ref = formula(X, A, B, scale, ids, dY)
    Wn = [w.double().cpu().numpy() for w in Ws]
    base = oracle.ks_chain_matmul(ps, Wn, X.double().cpu().numpy())
    back = dY.double().cpu().numpy()
    for p, w in zip(ps[::-1], Wn[::-1]):
        back = oracle.ks_matmul_dx(p, w, back)
    for got, want in ((Y, torch.from_numpy(base) + ref["D"]), (dX, torch.from_numpy(back) + ref["dX"]),
                      (dA, ref["dA"]), (dB, ref["dB"])):
        err = float((got.double().cpu() - want).norm() / want.norm())
        assert err <= FP32_REL_TOL, err
    only = chain.backward(dY, X, H, ids, weights=False)
    assert torch.equal(only[0], dX) and only[1] is None and only[2] is None
    # with transposed blocks at hand: the same bits; after a change of W: its gradient
    ready = libks.AdapterChain(Ws, ps, A, B, scale, transposed=True)
    assert all(torch.equal(a, b) for a, b in zip(ready.backward(dY, X, H, ids), (dX, dA, dB)))
    Ws[0].mul_(-1.5)
    changed = ready.backward(dY, X, H, ids)[0]
    assert torch.equal(changed, chain.backward(dY, X, H, ids)[0]) and not torch.equal(changed, dX)


PAIR = [(1, 64, 16, 64), (64, 8, 8, 8)]


@pytest.mark.parametrize("rank,xt,mix,batch", [
    (16, BF16, "runs", 1025), (8, BF16, "random", 1026), (4, BF16, "runs", 4099), (12, BF16, "random", 4098), (16, BF16, "runs", 5001), (16, F32, "random", 4097),
    (20, F32, "runs", 4110), (32, BF16, "random", 4097), (32, BF16, "runs", 4999), (16, BF16, "none", 4100),
    (20, BF16, "runs", 1030), (28, BF16, "random", 1027), (13, BF16, "runs", 4100), (48, BF16, "runs", 4100)])
def test_pair_adds_adapters(rank, xt, mix, batch):
    """Many rows through the fused pair of factors, which adds the adapters itself
    where it can: against 64 bits, rows of several adapters in a tile, NaN in the
    adapters of other rows."""
    require_gpu()
    X, A, B, scale, ids = draw(batch, 1024, 4096, 6, rank, xt, BF16, seed=rank + batch, mix=mix)
    ids[ids == 4] = 3
    A[4], B[4] = float("nan"), float("inf")                  # of no row
    A[5], B[5] = float("nan"), float("nan")
    Ws = [(torch.randn(a, d, b, c) / c ** 0.5).to(BF16).to(DEV) for a, b, c, d in PAIR]
    chain = libks.AdapterChain(Ws, PAIR, A, B, scale)
    Y, H = chain.matmul(X, ids, keep=True)
    assert torch.equal(Y.view(torch.int32), chain.matmul(X, ids).view(torch.int32))
    bad = ids == 5
    assert not torch.isfinite(Y[bad]).any() and torch.isfinite(Y[~bad]).all()
    A[4:], B[4:] = 0.0, 0.0
    ok = ~bad
    ref = formula(X[ok], A, B, scale, ids[ok])
    mag = formula(X[ok].abs(), A.abs(), B.abs(), scale, ids[ok])
    near(H[ok], ref["H"], mag["H"], 1024 + 2, "H")
    Wn, x = [w.double().cpu().numpy() for w in Ws], X[ok].double().cpu().numpy()
    base = torch.from_numpy(oracle.ks_chain_matmul(PAIR, Wn, x))
    size = torch.from_numpy(oracle.ks_chain_matmul(PAIR, [abs(w) for w in Wn], abs(x)))
    near(Y[ok], base + ref["D"], size + mag["D"], 1024 + rank + 26 + 4, "Y")


@pytest.mark.parametrize("b0,batch,xt,shift", [(64, 1, BF16, 0), (64, 3, F32, 0), (64, 1027, BF16, 0), (48, 70, BF16, 0),
                                               (32, 2050, F32, 0), (16, 9, BF16, 0), (80, 33, BF16, 0), (64, 21, BF16, 1)])
def test_gradient_of_the_pair(b0, batch, xt, shift):
    """dX of the fused pair's gradient, of other widths and of a dY that is not
    16-byte aligned, against 64 bits."""
    require_gpu()
    ps = [(1, b0, 16, 64), (b0, 8, 8, 8)]
    n_out = b0 * 64
    X, A, B, scale, ids = draw(batch, 1024, n_out, 2, 4, xt, BF16, seed=b0 + batch, mix="random")
    Ws = [(torch.randn(a, d, b, c) / c ** 0.5).to(BF16).to(DEV) for a, b, c, d in ps]
    chain = libks.AdapterChain(Ws, ps, A, B, scale)
    flat = torch.randn(batch * n_out + shift, device=DEV)
    dY = flat[shift:].view(batch, n_out)
    _, H = chain.matmul(X, ids, keep=True)
    dX = chain.backward(dY, X, H, ids)[0]
    assert torch.equal(dX, chain.backward(dY, X, H, ids)[0])
    ref, mag = formula(X, A, B, scale, ids, dY), formula(X.abs(), A.abs(), B.abs(), scale, ids, dY.abs())
    Wn = [w.double().cpu().numpy() for w in Ws]
    back, size = dY.double().cpu().numpy(), dY.double().cpu().abs().numpy()
    for p, w in zip(ps[::-1], Wn[::-1]):
        back, size = oracle.ks_matmul_dx(p, w, back), oracle.ks_matmul_dx(p, abs(w), size)
    near(dX, torch.from_numpy(back) + ref["dX"], torch.from_numpy(size) + mag["dX"], n_out + b0 + 8 + 4 + 4, "dX")


def test_layer_autograd_other_stream_and_graph():
    require_gpu()
    base = layer.KSLinear([(4, 64, 16, 6)], device=DEV, seed=3)
    m = layer.AdapterLinear(base, 4, 8, seed=1)
    x = torch.randn(2, 50, 384, device=DEV, requires_grad=True)
    ids = torch.tensor([2, -1], dtype=torch.int32, device=DEV)[:, None].expand(2, 50).contiguous()
    with torch.no_grad():
        # a new adapter changes nothing
        assert torch.equal(m(x, ids), libks.chain_matmul(x.detach().view(100, 384), list(base.weights),
                                                         base.patterns).view(2, 50, -1))
        m.B.normal_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = m(x, ids)
        y.square().sum().backward()
    torch.cuda.current_stream().wait_stream(side)
    assert x.grad.shape == x.shape and m.A.grad.abs().sum() > 0 and all(w.grad is None for w in base.weights)
    assert not m.A.grad[[0, 1, 3]].any()
    ref = formula(x.detach().view(100, 384), m.A, m.B, m.scale, ids.view(-1), 2 * y.detach().view(100, -1))
    assert float((m.A.grad.double().cpu() - ref["dA"]).norm() / ref["dA"].norm()) <= FP32_REL_TOL
    # a captured call, replayed with eager work in between
    chain = libks.AdapterChain(list(base.weights), base.patterns, m.A.detach(), m.B.detach(), m.scale)
    for batch in (16, 1300):
        X = torch.randn(batch, 384, device=DEV)
        who = torch.arange(batch, device=DEV, dtype=torch.int32) % 5
        out = torch.empty(batch, 1536, device=DEV)
        chain.matmul(X, who, out=out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            chain.matmul(X, who, out=out)
        for k in range(4):
            X.normal_()
            who.copy_((torch.arange(batch, device=DEV) * (k + 3)) % 6)
            want = chain.matmul(X, who)
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)


def test_batches_whose_output_passes_4_gib():
    require_gpu()
    batch, n_in, n_out = 270_001, 64, 4096
    g = torch.Generator(device=DEV).manual_seed(1)
    X = torch.randn(batch, n_in, device=DEV, generator=g)
    A = torch.randn(2, 4, n_in, device=DEV, generator=g)
    B = torch.randn(2, n_out, 4, device=DEV, generator=g)
    scale = torch.ones(2, device=DEV)
    ids = (torch.arange(batch, device=DEV) // 1000 % 3).to(torch.int32)
    out = torch.zeros(batch, n_out, device=DEV)
    Y, H = libks.adapter_matmul(X, A, B, scale, ids, out, keep=True)
    rows = torch.tensor([0, 999, 1000, 131_071, 131_072, 262_143, 262_145, batch - 1], device=DEV)
    ref = formula(X[rows], A, B, scale, ids[rows])
    mag = formula(X[rows].abs(), A.abs(), B.abs(), scale, ids[rows])
    near(Y[rows], ref["D"], mag["D"], n_in + 8, "Y")
    dX = torch.zeros(batch, n_in, device=DEV)
    libks.adapter_backward(Y, X, H, A, B, scale, ids, dX=dX)
    back = formula(X[rows], A, B, scale, ids[rows], Y[rows])
    bmag = formula(X[rows].abs(), A.abs(), B.abs(), scale, ids[rows], Y[rows].abs())
    near(dX[rows], back["dX"], bmag["dX"], n_out + 8, "dX")


def test_pair_on_another_stream_and_in_a_graph():
    """The fused pair with adapters and its gradient: bits of the call on the default
    stream, from another stream and from replays of a graph with eager work between."""
    require_gpu()
    batch = 1410
    X, A, B, scale, ids = draw(batch, 1024, 4096, 5, 16, BF16, BF16, seed=3, mix="runs")
    Ws = [(torch.randn(a, d, b, c) / c ** 0.5).to(BF16).to(DEV) for a, b, c, d in PAIR]
    chain = libks.AdapterChain(Ws, PAIR, A, B, scale)
    dY = torch.randn(batch, 4096, device=DEV)

    def both():
        Y, H = chain.matmul(X, ids, keep=True)
        return (Y, H) + chain.backward(dY, X, H, ids)

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for k in range(4):
        X.normal_()
        dY.normal_()
        ids.copy_(((torch.arange(batch, device=DEV) + 37 * k) // (50 + k)) % 6)
        want = both()
        for t in held:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_pair_past_32_bit_offsets():
    """The fused pair with adapters and its gradient where Y and dY pass 4 GiB."""
    require_gpu()
    batch = 270_003
    g = torch.Generator(device=DEV).manual_seed(1)
    X = torch.randn(batch, 1024, device=DEV, generator=g, dtype=BF16)
    A = (torch.randn(3, 8, 1024, device=DEV, generator=g) / 32).to(BF16)
    B = torch.randn(3, 4096, 8, device=DEV, generator=g).to(BF16)
    Ws = [(torch.randn(a, d, b, c) / c ** 0.5).to(BF16).to(DEV) for a, b, c, d in PAIR]
    scale = torch.ones(3, device=DEV)
    ids = (torch.arange(batch, device=DEV) // 1001 % 4).to(torch.int32)
    chain = libks.AdapterChain(Ws, PAIR, A, B, scale)
    Y, H = chain.matmul(X, ids, keep=True)
    dX = chain.backward(Y, X, H, ids, weights=False)[0]
    # the same rows in a short batch of their own: the neighbours of a row do not matter
    for n0 in (0, 131_064, 262_136, batch - 1203):
        rows = slice(n0, n0 + 1203)
        Ys, Hs = chain.matmul(X[rows].clone(), ids[rows].clone(), keep=True)
        dXs = chain.backward(Y[rows].clone(), X[rows].clone(), Hs, ids[rows].clone(), weights=False)[0]
        for whole, part in ((Y[rows], Ys), (H[rows], Hs), (dX[rows], dXs)):
            assert float((whole.double() - part.double()).norm() / part.double().norm()) <= FP32_REL_TOL
