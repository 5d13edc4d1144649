"""AdamW over many tensors (needs an MI355X) against the formula in 64 bits,
and its 8-bit moments against the same fp32 arithmetic in numpy.

Tolerances. m = b1 m + c1 g is two rounded products and a rounded sum: within
3 2^-24 of |b1 m| + |c1 g|, and v likewise with one product more; constants
rounded to fp32 add 2^-24 each. p = decay p - rate m / root: its own rounding
(2^-23 |p|), and of the update the errors of m and of root (sqrt and reciprocal
to 1 ulp each, v's error halved): 8 2^-23 of it beside m's.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from gpu_helpers import DEV, require_gpu
from kronecker_sparse_structured_amd import libks, optim

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
H = dict(lr=2e-3, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)
SIZES = [1, 7, 255, 256, 257, 1023, 4096, 4097, 65536, 100001]


def tensors(sizes, pt, gt, seed, offset=0):
    g = torch.Generator().manual_seed(seed)

    def make(scale, t, positive=False):
        out = []
        for n in sizes:
            x = torch.randn(n + offset, generator=g) * scale
            out.append((x.abs() if positive else x).to(t).to(DEV)[offset:])
        return out

    return make(0.3, pt), make(0.05, gt), make(0.01, F32), make(1e-3, F32, True)


def formula(p, g, m, v, step, scale=1.0):
    p, g, m, v = (t.double().cpu() for t in (p, g, m, v))
    b1, b2 = H["betas"]
    g = g * scale
    m2, v2 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    root = (v2 / (1 - b2 ** step)).sqrt() + H["eps"]
    upd = H["lr"] / (1 - b1 ** step) * m2 / root
    mm = b1 * m.abs() + (1 - b1) * g.abs()
    bound_m = 5 * 2.0 ** -24 * mm
    bound_v = 7 * 2.0 ** -24 * v2
    bound_p = 2.0 ** -23 * p.abs() + H["lr"] / (1 - b1 ** step) * (bound_m + 8 * 2.0 ** -23 * m2.abs()) / root
    return p - H["lr"] * H["weight_decay"] * p - upd, m2, v2, bound_p, bound_m, bound_v


def assert_within(got, want, bound, what):
    err = (got.double().cpu() - want).abs()
    assert bool((err <= bound + 1e-37).all()), "%s: %g" % (what, float((err / (bound + 1e-37)).max()))


@pytest.mark.parametrize("pt,gt", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("offset", [0, 1])
def test_step_in_32_bits(pt, gt, offset):
    require_gpu()
    ps, gs, ms, vs = tensors(SIZES, pt, gt, seed=offset + 1, offset=offset)
    want = [formula(p, g, m, v, 3) for p, g, m, v in zip(ps, gs, ms, vs)]
    libks.AdamW(ps, gs, ms, vs).step(3, **H)
    for p, m, v, w in zip(ps, ms, vs, want):
        assert_within(m, w[1], w[4], "m")
        assert_within(v, w[2], w[5], "v")
        assert_within(p, w[0], w[3] + (w[0].abs() * 2.0 ** -8 if pt == BF16 else 0), "p")


def test_more_tensors_than_a_launch_takes_and_empty_ones():
    require_gpu()
    sizes = [37 + 11 * i for i in range(150)] + [0, 5, 0]
    ps, gs, ms, vs = tensors(sizes, F32, F32, seed=5)
    want = [formula(p, g, m, v, 1) for p, g, m, v in zip(ps, gs, ms, vs)]
    libks.AdamW(ps, gs, ms, vs).step(1, **H)
    for p, m, v, w in zip(ps, ms, vs, want):
        assert_within(p, w[0], w[3], "p")
        assert_within(m, w[1], w[4], "m")
        assert_within(v, w[2], w[5], "v")
    libks.AdamW([], [], [], []).step(1, **H)


def test_norm_and_clip():
    require_gpu()
    for gt in (F32, BF16):
        ps, gs, ms, vs = tensors(SIZES + [300000], F32, gt, seed=7)
        opt = libks.AdamW(ps, gs, ms, vs)
        want = math.sqrt(sum(float(g.double().square().sum()) for g in gs))
        norm = opt.grad_norm()
        # 16384 squares at most to a workgroup, the rest in double
        assert abs(float(norm) - want) <= 80 * 2.0 ** -24 * want
        assert torch.equal(norm, opt.grad_norm())
        ref = [formula(p, g, m, v, 2, scale=min(1.0, 0.5 / (want + 1e-6))) for p, g, m, v in zip(ps, gs, ms, vs)]
        assert float(opt.step(2, max_norm=0.5, **H)) == float(norm)
        for p, m, v, w in zip(ps, ms, vs, ref):
            # the scale is off by the norm's error
            assert_within(p, w[0], w[3] * 40, "p")
            assert_within(m, w[1], w[4] * 40, "m")
        # a bound above the norm changes nothing
        a = [t.clone() for t in ps]
        opt.step(2, max_norm=1e9, **H)
        ps2, gs2, ms2, vs2 = a, gs, *tensors(SIZES + [300000], F32, gt, seed=7)[2:]
        assert len(ps2) == len(vs2)


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_norm_that_is_not_finite_changes_nothing(bits, bad):
    require_gpu()
    ps, gs, ms, vs = tensors([300, 5000], F32, F32, seed=9)
    scales = None
    if bits == 8:
        ms, vs, scales = encoded(ms, vs)
    gs[1][17] = bad
    before = [t.clone() for t in (*ps, *ms, *vs, *(scales or ()))]
    libks.AdamW(ps, gs, ms, vs, scales).step(1, max_norm=1.0, **H)
    assert all(torch.equal(a, b) for a, b in zip(before, (*ps, *ms, *vs, *(scales or ()))))


# ---------------------------------------------------------------- 8 bits

f = np.float32
TOP_M, TOP_V = f(127.0 ** 2), f(255.0 ** 4)


def blocks(x):
    out = np.zeros(-(-len(x) // 256) * 256, dtype=x.dtype)
    out[:len(x)] = x
    return out.reshape(-1, 256)


def value_m(k, s):
    k = blocks(k.astype(f))
    return (k * np.abs(k)) * (s[:, None] * (f(1) / TOP_M))


def value_v(k, s):
    k = blocks(k.astype(f))
    return ((k * k) * (k * k)) * (s[:, None] * (f(1) / TOP_V))


def random_bits(n, base, seed):
    x = ((np.arange(n, dtype=np.uint64) + base) * 0x9E3779B1 + seed) & 0xFFFFFFFF
    x ^= x >> 16
    x = (x * 0xAADDE6A9) & 0xFFFFFFFF
    x ^= x >> 15
    x = (x * 0xBEDE544D) & 0xFFFFFFFF
    return x ^ (x >> 16)


def code_m(m, chance):
    s = np.maximum(np.abs(m).max(1), f(1e-30))
    u = np.abs(m) * ((f(1) / s) * TOP_M)[:, None]
    k = np.minimum(np.floor(np.sqrt(u)), f(127))
    k = np.minimum(k + (chance * (f(2) * k + f(1)) < u - k * k), f(127))
    return (np.sign(m) * k).astype(np.int8), s


def code_v(v, chance):
    s = np.maximum(v.max(1), f(1e-28))
    u = v * ((f(1) / s) * TOP_V)[:, None]
    k = np.minimum(np.floor(np.sqrt(np.sqrt(u))), f(255))
    low, high = (k * k) * (k * k), ((k + f(1)) * (k + f(1))) * ((k + f(1)) * (k + f(1)))
    k = k + (chance * (high - low) < u - low)
    k = np.where((k < 1) & (v > 0), f(1), k)
    return np.minimum(k, f(255)).astype(np.uint8), s


def encoded(ms, vs):
    """8-bit states near the given moments (rounded down)."""
    out_m, out_v, scales = [], [], []
    for m, v in zip(ms, vs):
        n = m.numel()
        full = np.full((-(-n // 256), 256), f(0.999))
        km, sm = code_m(blocks(m.cpu().numpy()), full)
        kv, sv = code_v(blocks(v.cpu().numpy()), full)
        out_m.append(torch.from_numpy(km.reshape(-1)[:n].copy()).to(DEV))
        out_v.append(torch.from_numpy(kv.reshape(-1)[:n].copy()).to(DEV))
        scales.append(torch.from_numpy(np.stack([sm, sv], 1).astype(f)).to(DEV))
    return out_m, out_v, scales


def model_step(m, v, s, g, base, seed):
    """codes and scales after a step, in fp32 one operation at a time"""
    n = len(m)
    b1, b2 = f(H["betas"][0]), f(H["betas"][1])
    c1, c2 = f(1 - H["betas"][0]), f(1 - H["betas"][1])
    g = blocks(g)
    m = value_m(m, s[:, 0]) * b1 + g * c1
    v = value_v(v, s[:, 1]) * b2 + (g * g) * c2
    bits = random_bits(m.size, base, seed).reshape(m.shape)
    km, sm = code_m(m, (bits & 0xFFFF).astype(f) / f(65536))
    kv, sv = code_v(v, (bits >> 16).astype(f) / f(65536))
    return m, v, km.reshape(-1)[:n], kv.reshape(-1)[:n], np.stack([sm, sv], 1)


@pytest.mark.parametrize("pt,gt,offset", [(F32, F32, 0), (BF16, BF16, 0), (F32, BF16, 1), (BF16, F32, 3)])
def test_step_in_8_bits(pt, gt, offset):
    require_gpu()
    ps, gs, ms, vs = tensors(SIZES, pt, gt, seed=offset + 11, offset=offset)
    ms, vs, scales = encoded(ms, vs)
    if offset:
        ms = [torch.cat([t[:1].expand(offset), t])[offset:] for t in ms]
    want, base = [], 0
    for p, g, m, v, s in zip(ps, gs, ms, vs, scales):
        host = [t.float().cpu().numpy() if t.dtype == BF16 else t.cpu().numpy() for t in (m, v, s, g)]
        mw, vw, km, kv, sw = model_step(*host, base, 99)
        n = p.numel()
        wide = formula(p, g, torch.from_numpy(value_m(host[0], host[2][:, 0]).reshape(-1)[:n].copy()),
                       torch.from_numpy(value_v(host[1], host[2][:, 1]).reshape(-1)[:n].copy()), 5)
        want.append((km, kv, sw, wide))
        base += -(-n // 256) * 256
    opt = libks.AdamW(ps, gs, ms, vs, scales)
    opt.step(5, seed=99, **H)
    mo = [torch.empty(p.numel(), device=DEV) for p in ps]
    vo = [torch.empty(p.numel(), device=DEV) for p in ps]
    opt.state_values(mo, vo)
    for p, m, v, s, a, b, (km, kv, sw, wide) in zip(ps, ms, vs, scales, mo, vo, want):
        assert np.array_equal(s.cpu().numpy(), sw)
        assert np.array_equal(m.cpu().numpy(), km) and np.array_equal(v.cpu().numpy(), kv)
        assert np.array_equal(a.cpu().numpy(), value_m(km, sw[:, 0]).reshape(-1)[:len(km)])
        assert np.array_equal(b.cpu().numpy(), value_v(kv, sw[:, 1]).reshape(-1)[:len(kv)])
        assert_within(p, wide[0], wide[3] * 2 + (wide[0].abs() * 2.0 ** -8 if pt == BF16 else 0), "p")


def test_rounding_keeps_the_mean_and_v_can_fall():
    """400 steps without gradients: v falls by b2 each step, which is less than
    half a code. The mean over 4096 values of a walk whose steps keep the mean
    is within 5 standard errors; a step's spread is at most a code, 4 / k of the
    value with k >= 100 here."""
    require_gpu()
    n, steps, b2 = 4096, 400, 0.999
    p, g = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    m = torch.zeros(n, dtype=torch.int8, device=DEV)
    v = torch.full((n,), 200, dtype=torch.uint8, device=DEV)
    v[::256] = 255
    s = torch.ones(n // 256, 2, device=DEV)
    opt = libks.AdamW([p], [g], [m], [v], [s])
    out = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
    opt.state_values([out[0]], [out[1]])
    keep = torch.ones(n, dtype=torch.bool, device=DEV)
    keep[::256] = False
    start = float(out[1][keep].double().mean())
    for t in range(steps):
        opt.step(t + 1, lr=0.0, betas=(0.9, b2), weight_decay=0.0, seed=t * 7919 + 1)
    opt.state_values([out[0]], [out[1]])
    end = float(out[1][keep].double().mean())
    spread = (4 / 100) * start * 0.5 * math.sqrt(steps) / math.sqrt(n)
    assert abs(end - start * b2 ** steps) <= 5 * spread
    assert not m.any()


def test_values_that_are_not_finite_stay_in_their_block():
    require_gpu()
    ps, gs, ms, vs = tensors([1000], F32, F32, seed=3)
    ms, vs, scales = encoded(ms, vs)
    gs[0][300] = float("nan")
    opt = libks.AdamW(ps, gs, ms, vs, scales)
    opt.step(1, **H)
    ok = torch.isfinite(scales[0]).all(dim=1)
    assert ok.tolist() == [True, False, True, True]
    assert torch.isfinite(ps[0][:256]).all() and torch.isfinite(ps[0][512:]).all() and torch.isnan(ps[0][300])


def test_optimizer_class_state_dict_and_graph():
    require_gpu()
    for bits in (32, 8):
        torch.manual_seed(0)
        w = [torch.nn.Parameter(torch.randn(300, 7, device=DEV)), torch.nn.Parameter(torch.randn(33, device=DEV)),
             torch.nn.Parameter(torch.randn(5, device=DEV))]
        opt = optim.AdamW([{"params": w[:2]}, {"params": w[2:], "lr": 5e-2}], lr=1e-2, state_bits=bits, max_norm=3.0,
                          seed=5)
        first = None
        for _ in range(30):
            opt.zero_grad()
            loss = sum((p - 1).square().sum() for p in w)
            loss.backward()
            opt.step()
            first = first if first is not None else float(loss)
        assert float(loss) < first
        saved = opt.state_dict()
        twin = [torch.nn.Parameter(p.detach().clone()) for p in w]
        other = optim.AdamW([{"params": twin[:2]}, {"params": twin[2:], "lr": 5e-2}], lr=1e-2, state_bits=bits,
                            max_norm=3.0, seed=5)
        other.load_state_dict(saved)
        for a, b in zip(w, twin):
            a.grad = torch.ones_like(a)
            b.grad = torch.ones_like(b)
        opt.step()
        other.step()
        assert all(torch.equal(a, b) for a, b in zip(w, twin))
    ps, gs, ms, vs = tensors([5000, 77], F32, F32, seed=2)
    opt = libks.AdamW(ps, gs, ms, vs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        opt.step(1, max_norm=0.1, **H)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step(1, max_norm=0.1, **H)
    for _ in range(4):
        for g in gs:
            g.normal_()
        start = [[t.clone() for t in ts] for ts in (ps, ms, vs)]
        graph.replay()
        torch.cuda.synchronize()
        got = [[t.clone() for t in ts] for ts in (ps, ms, vs)]
        for ts, ss in zip((ps, ms, vs), start):
            for t, x in zip(ts, ss):
                t.copy_(x)
        opt.step(1, max_norm=0.1, **H)
        assert all(torch.equal(a, b) for x, y in zip(got, (ps, ms, vs)) for a, b in zip(x, y))


def test_refusals():
    require_gpu()
    ps, gs, ms, vs = tensors([16], F32, F32, seed=1)
    with pytest.raises(ValueError):
        libks.AdamW(ps, [], ms, vs)
    with pytest.raises(ValueError):
        libks.AdamW(ps, gs, ps, vs)
    with pytest.raises(TypeError):
        libks.AdamW(ps, gs, ms, vs, [torch.zeros(1, 2, device=DEV)])
    with pytest.raises(libks.KSError):
        libks.AdamW(ps, gs, ms, vs).step(0, **H)
    with pytest.raises(ValueError):
        libks.AdamW(ps, gs, ms, vs).step(1, max_norm=0.0, **H)
    with pytest.raises(ValueError):
        libks.AdamW(ps, gs, ms, vs).state_values([ms[0]], [vs[0]])
