"""The norms around a block with its gate and residual (needs an MI355X) against
the formulas in 64 bits.

Tolerances, with u = 2^-24. A sum over a row of width D is formed from at most 8
values a lane, 6 exchanges and 16 waves: 30 roundings of its terms' magnitudes;
everything around it takes a handful more. So with N = 64:
* the normed value n = (v - mean) r is off by at most N u A (1 + |n|), where
  A = r max (|v| + mean |v|) over the row is what the difference from the mean
  can lose (r changes by r^2 times what the values change), plus r times what
  v itself is off by, twice (it moves the mean and r as well);
* a product of such values by the product of magnitudes, times the sum of the
  relative errors;
* a sum over rows by the rows' bounds, plus (rows / 512 + 64) u of its terms'
  magnitudes (a worker's part and the workers of a workgroup; the rest is double);
* a result in bf16 is rounded once: 2^-8 of it (half a step), with the error
  before it.
"""
from __future__ import annotations

import pytest
import torch

from gpu_helpers import DEV, require_gpu
from kronecker_sparse_structured_amd import libks

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
U, N = 2.0 ** -24, 64
VECTORS = ("pre_weight", "pre_bias", "post_weight", "post_bias", "scale")


def make(rows, width, kind="rms", pre=True, post=True, bias=True, scale=True, groups=0, x=F32, y=F32, h=F32, params=F32,
         gate=F32, seed=0, residual=0.7, eps=1e-5):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g)

    have = {"pre_weight": pre, "pre_bias": pre and bias, "post_weight": post, "post_bias": post and bias, "scale": scale}
    p = {"kind": kind, "eps": eps, "residual": residual, "h": h, "width": width, "groups": groups}
    p["x"] = (2 * normal(rows, width) + 1).to(x).to(DEV)
    p["y"] = None if y is None else ((0.5 + torch.rand(rows, 1, generator=g)) * normal(rows, width) - 0.3).to(y).to(DEV)
    p["gate"] = (1 + 0.5 * normal(groups, width)).to(gate).to(DEV) if groups else None
    p["vectors"] = {k: (("bias" not in k) + 0.3 * normal(width)).to(params).to(DEV) if on else None
                    for k, on in have.items()}
    p["dz"] = normal(rows, width).to(x).to(DEV)
    p["dh"] = normal(rows, width).to(h).to(DEV) if pre else None
    return p


def handle(p):
    return libks.ResidualNorm(p["width"], **p["vectors"], kind=p["kind"], eps=p["eps"], residual=p["residual"])


def formula(p):
    """(values, bounds) of every output, in 64 bits on the CPU."""
    wide = {k: None if t is None else t.double().cpu() for k, t in
            {**p["vectors"], "x": p["x"], "y": p["y"], "gate": p["gate"], "dz": p["dz"], "dh": p["dh"]}.items()}
    x, y, dz, dh = (wide[k] for k in ("x", "y", "dz", "dh"))
    rows, D = x.shape
    layer = p["kind"] == "layer"
    zero = torch.zeros_like(x)

    def norm(v, dv):
        mean = v.mean(1, keepdim=True) if layer else torch.zeros(rows, 1, dtype=torch.float64)
        r = 1 / torch.sqrt((v - mean).square().mean(1, keepdim=True) + p["eps"])
        n = (v - mean) * r
        A = r * (v.abs() + v.abs().mean(1, keepdim=True)).amax(1, keepdim=True) if D else r
        return n, r, N * U * A * (1 + n.abs()) + 2 * r * (dv + dv.amax(1, keepdim=True) * (1 + n.abs()))

    def vec(k, default):
        return torch.full((D,), default, dtype=torch.float64) if wide[k] is None else wide[k]

    w1, b1, w2, b2, s = vec("pre_weight", 0.0), vec("pre_bias", 0.0), vec("post_weight", 1.0), vec("post_bias", 0.0), \
        vec("scale", 1.0)
    gate = torch.ones(1, 1, dtype=torch.float64)
    if p["gate"] is not None:
        gate = wide["gate"].repeat_interleave(rows // p["groups"], 0) if rows else torch.ones_like(x)
    c = p["residual"]
    val, tol = {}, {}
    post = wide["post_weight"] is not None and y is not None
    z, ez = x, zero
    if y is not None:
        yn, r2, eyn = norm(y, zero) if post else (y, torch.ones(rows, 1, dtype=torch.float64), zero)
        uu = yn * w2 + b2
        eu = eyn * w2.abs() + 4 * U * (yn.abs() * w2.abs() + b2.abs())
        add = c * s * gate * uu
        z = x + add
        ez = (c * s * gate).abs() * eu + 8 * U * (add.abs() + x.abs())
        val["z"], tol["z"] = z, ez
    zn, r1, ezn = norm(z, ez)
    if wide["pre_weight"] is not None:
        val["h"] = zn * w1 + b1
        tol["h"] = ezn * w1.abs() + 4 * U * (zn.abs() * w1.abs() + b1.abs())
    # gradients
    dn = dh * w1 if dh is not None else zero
    znm, ezm = zn.abs(), ezn
    D1 = max(D, 1)

    def back(d, ed, n, en, r, er):
        """d behind a norm, and its bound; er is r's relative error."""
        A, B = (d * n).sum(1, keepdim=True) / D1, d.sum(1, keepdim=True) / D1
        Am, Bm = (d * n).abs().sum(1, keepdim=True) / D1, d.abs().sum(1, keepdim=True) / D1
        eA = (ed * n.abs() + d.abs() * en).sum(1, keepdim=True) / D1 + N * U * Am
        eB = ed.sum(1, keepdim=True) / D1 + N * U * Bm
        out = r * (d - n * A - (B if layer else 0.0))
        size = d.abs() + n.abs() * Am + (Bm if layer else 0.0)
        e = r * (ed + n.abs() * eA + en * Am + (eB if layer else 0.0)) + (er + 8 * U) * r * size
        return out, e

    er1 = r1 * 2 * ez.amax(1, keepdim=True) * 2 + N * U * (1 + r1 * z.abs().mean(1, keepdim=True)) if D else r1
    dx, edx = (dz if dz is not None else zero), zero
    if dh is not None:
        t, e = back(dn, 2 * U * dn.abs(), zn, ezn, r1, er1)
        dx, edx = dx + t, e + 2 * U * (dx.abs() + t.abs())
    val["dx"], tol["dx"] = dx, edx
    count = (rows / 512 + 64) * U

    def over_rows(v, e):
        return v.sum(0), e.sum(0) + count * v.abs().sum(0)

    if dh is not None:
        val["pre_weight"], tol["pre_weight"] = over_rows(dh * zn, dh.abs() * ezn)
        val["pre_bias"], tol["pre_bias"] = over_rows(dh, zero)
    elif wide["pre_weight"] is not None:
        val["pre_weight"] = val["pre_bias"] = tol["pre_weight"] = tol["pre_bias"] = torch.zeros(D, dtype=torch.float64)
    if y is not None:
        t, et = c * dx, abs(c) * edx + 2 * U * (c * dx).abs()
        du = t * s * gate
        edu = (s * gate).abs() * et + 4 * U * du.abs()
        val["post_weight"], tol["post_weight"] = over_rows(du * yn, edu * yn.abs() + du.abs() * eyn)
        val["post_bias"], tol["post_bias"] = over_rows(du, edu)
        ds = t * gate * uu
        eds = gate.abs() * (et * uu.abs() + t.abs() * eu) + 4 * U * ds.abs()
        val["scale"], tol["scale"] = over_rows(ds, eds)
        if p["gate"] is not None:
            dg = t * s * uu
            edg = s.abs() * (et * uu.abs() + t.abs() * eu) + 4 * U * dg.abs()
            k = rows // p["groups"]
            val["gate"] = dg.view(p["groups"], k, D).sum(1)
            tol["gate"] = edg.view(p["groups"], k, D).sum(1) + (k / 8 + 64) * U * dg.abs().view(p["groups"], k, D).sum(1)
        dm, edm = du * w2, edu * w2.abs() + 2 * U * (du * w2).abs()
        if post:
            er2 = N * U * (1 + r2 * y.abs().mean(1, keepdim=True)) if D else r2
            val["dy"], tol["dy"] = back(dm, edm, yn, eyn, r2, er2)
        else:
            val["dy"], tol["dy"] = du, edu
    return val, tol


def check(p, got, want=None, names=None):
    val, tol = want or formula(p)
    for k, t in got.items():
        if t is None or (names and k not in names):
            continue
        v, e = val[k], tol[k].clone() + 1e-30
        assert tuple(t.shape) == tuple(v.shape), k
        if t.dtype == BF16:
            e = e * (1 + 2.0 ** -7) + v.abs() * 2.0 ** -8
        else:
            e = e + v.abs() * U
        err = (t.double().cpu() - v).abs()
        assert bool((err <= e).all()), "%s: %g of its bound" % (k, float((err / e).max()))


def run(p, dz=True, dh=True, weights=True, stream=None):
    n = handle(p)
    z, h, stats = n.forward(p["x"], p["y"], p["gate"], dtype=p["h"], keep=True, stream=stream)
    g = n.backward(p["dz"] if dz else None, p["dh"] if dh else None, p["x"], p["y"], stats, p["gate"], weights=weights,
                   stream=stream)
    out = {"h": h, **g._asdict()}
    if p["y"] is not None:
        out["z"] = z
    for k in VECTORS:
        assert (out[k] is None) == (p["vectors"][k] is None or not weights)
    return out


SIZES = [(1, 1), (3, 7), (5, 8), (2, 63), (17, 384), (1, 512), (9, 513), (33, 1000), (7, 1024), (130, 1023), (3, 4096),
         (2, 4100), (5, 8192), (2, 8191), (700, 40)]


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "%dx%d" % s)
def test_every_output(size, kind):
    require_gpu()
    rows, width = size
    p = make(rows, width, kind, groups=rows, seed=rows + width)
    got = run(p)
    check(p, got)
    again = run(p)
    assert all(torch.equal(a, b) for a, b in zip(got.values(), again.values()))
    n = handle(p)
    z, h = n.forward(p["x"], p["y"], p["gate"], dtype=p["h"])
    assert torch.equal(z, got["z"]) and torch.equal(h, got["h"])


TYPES = [(a, b, c, d, e) for a in (F32, BF16) for b in (F32, BF16) for c in (F32, BF16) for d, e in
         ((F32, BF16), (BF16, F32))]


@pytest.mark.parametrize("width", [96, 333])
@pytest.mark.parametrize("types", TYPES, ids=lambda t: "-".join(str(v)[6:] for v in t))
def test_types(types, width):
    require_gpu()
    x, y, h, params, gate = types
    p = make(12, width, "layer", groups=3, x=x, y=y, h=h, params=params, gate=gate, seed=width)
    got = run(p)
    assert got["z"].dtype == got["dx"].dtype == x and got["dy"].dtype == y and got["h"].dtype == h
    assert got["gate"].dtype == gate and got["scale"].dtype == F32
    check(p, got)


@pytest.mark.parametrize("groups", [1, 2, 5, 100, 700, 3500])
@pytest.mark.parametrize("width", [64, 1000, 2048])
def test_gates_of_any_share(groups, width):
    require_gpu()
    p = make(3500, width, "rms", groups=groups, seed=groups)
    check(p, run(p))


def test_many_rows_a_worker():
    require_gpu()
    for rows, width, groups in ((20001, 32, 0), (20000, 32, 4), (20000, 32, 5000), (9000, 520, 0)):
        p = make(rows, width, "layer", groups=groups, seed=rows)
        check(p, run(p))


@pytest.mark.parametrize("groups", [0, 2, 300, 600])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_widest_rows(kind, groups):
    """More rows than workers where a row takes 16 waves of 8 values a lane."""
    require_gpu()
    for width, y in ((5001, F32), (8192, BF16)):
        p = make(600, width, kind, groups=groups, y=y, seed=groups + width)
        check(p, run(p))


PARTS = [dict(post=False), dict(scale=False), dict(bias=False), dict(pre=False), dict(pre=False, post=False),
         dict(post=False, scale=False, groups=0), dict(y=None, post=False, scale=False), dict(y=None)]


@pytest.mark.parametrize("part", PARTS, ids=lambda d: "-".join("%s=%s" % i for i in d.items()))
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_without_parts(part, kind):
    require_gpu()
    opts = {"groups": 0 if "y" in part else 2, **part}
    for width in (72, 1001):
        p = make(6, width, kind, seed=5, **opts)
        got = run(p)
        want = formula(p)
        if "y" in part:                      # vectors that nothing went through
            want[0].update({k: torch.zeros(width).double() for k in ("post_weight", "post_bias", "scale")})
            want[1].update({k: torch.zeros(width).double() for k in ("post_weight", "post_bias", "scale")})
        check(p, got, want)
        if "y" in part:
            z, h = handle(p).forward(p["x"], dtype=p["h"])
            assert z is p["x"] and torch.equal(h, got["h"])


def test_gradients_of_one_output_only():
    require_gpu()
    for dz, dh in ((True, False), (False, True), (False, False)):
        p = make(9, 200, "layer", groups=3, seed=2)
        got = run(p, dz=dz, dh=dh)
        q = dict(p, dz=p["dz"] if dz else torch.zeros_like(p["dz"]), dh=p["dh"] if dh else torch.zeros_like(p["dh"]))
        check(q, got)
    got = run(p, weights=False)
    assert all(got[k] is None for k in VECTORS) and got["gate"] is not None


def test_no_rows():
    require_gpu()
    p = make(0, 24, "layer", groups=0, seed=1)
    got = run(p)
    assert got["z"].shape == got["dx"].shape == (0, 24)
    assert all(not got[k].any() for k in VECTORS)
    n = handle(p)
    gate = torch.ones(3, 24, device=DEV)
    z, h, stats = n.forward(p["x"], p["y"], gate, keep=True)
    g = n.backward(p["dz"], p["dh"], p["x"], p["y"], stats, gate)
    assert g.gate.shape == (3, 24) and not g.gate.any()


def test_large_means_and_far_values():
    """A mean 1000 times the deviation: the difference of sums would lose it."""
    require_gpu()
    p = make(4, 640, "layer", groups=0, seed=9)
    p["x"] = p["x"] * 0.01 + 10.0
    p["y"] = p["y"] * 1e-3 + 1.0
    check(p, run(p))
    p["y"][1] = 0.0                                   # a row without a deviation
    p["x"][2] = 1e15
    p["x"][3] = 1e-20
    p["y"][3] = -1e-20
    got = run(p)
    for k in ("z", "h", "dx", "dy"):
        assert torch.isfinite(got[k]).all(), k


def test_infinities_and_nan_stay_in_their_rows():
    require_gpu()
    for width in (64, 1000):
        p = make(8, width, "layer", groups=8, seed=4)
        want = formula(p)
        p["x"][1, 3] = float("nan")
        p["y"][2, 5] = float("inf")
        p["dh"][5, 0] = float("nan")
        got = run(p)
        clean = [0, 3, 4, 6, 7]
        for k in ("z", "h", "dx", "dy", "gate"):
            v, e = want[0][k][clean], want[1][k][clean] + want[0][k][clean].abs() * U + 1e-30
            assert bool(((got[k][clean].double().cpu() - v).abs() <= e).all()), k
        assert torch.isnan(got["h"][1]).all() and torch.isnan(got["h"][2]).any() and torch.isnan(got["dx"][5]).all()


def test_unaligned_rows():
    require_gpu()
    for off in (1, 2, 3):
        p = make(5, 512, "rms", groups=5, x=BF16, y=F32, h=BF16, seed=off)
        want = formula(p)
        for k in ("x", "y", "dz", "dh", "gate"):
            buf = torch.empty(p[k].numel() + 8, dtype=p[k].dtype, device=DEV)
            buf[off:off + p[k].numel()] = p[k].reshape(-1)
            p[k] = buf[off:off + p[k].numel()].view(p[k].shape)
        check(p, run(p), want)


def test_differences():
    """The gradients against differences of the 64-bit formulas."""
    require_gpu()
    for kind in ("rms", "layer"):
        p = make(4, 40, kind, groups=2, seed=6)
        got = run(p)
        names = {"x": "dx", "y": "dy", "gate": "gate", **{k: k for k in VECTORS}}
        g = torch.Generator().manual_seed(1)

        def loss(q):
            v, _ = formula(q)
            return float((v["z"] * p["dz"].double().cpu()).sum() + (v["h"] * p["dh"].double().cpu()).sum())

        for k, name in names.items():
            t = p["vectors"][k] if k in VECTORS else p[k]
            D = torch.randn(t.shape, generator=g).double()
            step, ends = 1e-5, []
            for sign in (1, -1):
                moved = (t.double().cpu() + sign * step * D)
                q = dict(p, vectors=dict(p["vectors"]))
                if k in VECTORS:
                    q["vectors"][k] = moved
                else:
                    q[k] = moved
                ends.append(loss(q))
            num = (ends[0] - ends[1]) / (2 * step)
            ana = got[name].double().cpu()
            # fp32 gradients (2^-16 of the sum of magnitudes) and the difference's own step^2 and rounding
            assert abs(num - float((ana * D).sum())) <= 2.0 ** -16 * float((ana * D).abs().sum()) + 1e-6, (kind, k)


def test_in_place_residual():
    """z in x's own memory, through the C entry point."""
    require_gpu()
    p = make(37, 392, "rms", groups=37, seed=3)
    want = formula(p)
    n = handle(p)._n
    n.x_elem = n.y_elem = n.h_elem = n.gate_elem = libks.ELEM_F32
    h = torch.empty_like(p["x"])
    st = libks.load().ks_residual_norm(n, p["x"].data_ptr(), p["y"].data_ptr(), p["gate"].data_ptr(), 37,
                                       p["x"].data_ptr(), h.data_ptr(), None, 37,
                                       torch.cuda.current_stream().cuda_stream)
    assert st == libks.KS_OK
    check(p, {"z": p["x"], "h": h}, want)


def test_graph_and_streams():
    require_gpu()
    p = make(300, 264, "layer", groups=3, x=BF16, h=BF16, seed=8)
    n = handle(p)
    side = torch.cuda.Stream()
    a = run(p)
    side.wait_stream(torch.cuda.current_stream())
    b = run(p, stream=side)
    side.synchronize()
    assert all(torch.equal(s, t) for s, t in zip(a.values(), b.values()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z, h, stats = n.forward(p["x"], p["y"], p["gate"], dtype=BF16, keep=True)
        g = n.backward(p["dz"], p["dh"], p["x"], p["y"], stats, p["gate"])
    for k in range(4):
        p["y"].normal_()
        p["dh"].normal_()
        want = run(p)
        for t in (z, h, g.dx, g.dy, g.gate, g.scale, g.pre_weight):
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(z, want["z"]) and torch.equal(h, want["h"])
        assert all(torch.equal(t, want[name]) for name, t in g._asdict().items()), k


def test_past_2_31_values():
    require_gpu()
    rows, width = 270_000, 8192
    x = torch.zeros(rows, width, dtype=BF16, device=DEV)
    some = torch.tensor([0, 1, 262_143, 262_144, rows - 1], device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    x[some] = torch.randn(5, width, device=DEV, generator=g).to(BF16)
    w = torch.randn(width, device=DEV, generator=g)
    n = libks.ResidualNorm(width, w, eps=1e-5)
    z, h = n.forward(x, x, dtype=BF16)
    p = {"x": x[some], "y": x[some], "gate": None, "dz": None, "dh": None, "kind": "rms", "eps": 1e-5, "residual": 1.0,
         "vectors": {**dict.fromkeys(VECTORS), "pre_weight": w}, "groups": 0}
    check(p, {"z": z[some], "h": h[some]})
    assert not z[2:262_143].any() and not h[262_145:rows - 1].any()


def test_refusals():
    require_gpu()
    x, w = torch.zeros(4, 16, device=DEV), torch.ones(16, device=DEV)
    for bad in (dict(pre_bias=w), dict(pre_weight=w[:8]), dict(kind="batch"), dict(pre_weight=w, scale=w.bfloat16()),
                dict(pre_weight=w.double())):
        with pytest.raises((ValueError, TypeError)):
            libks.ResidualNorm(16, **bad)
    n = libks.ResidualNorm(16, w, post_weight=w)
    z, h, stats = n.forward(x, x.clone(), keep=True)
    for args in ((x[:, :8],), (x, x[:2]), (x, x.t().contiguous().t()), (x.half(),), (x, None, x[:1]), (x, x, x[:3]),
                 (x, x, x[:, :8].contiguous()), (x.cpu(),)):
        with pytest.raises((ValueError, TypeError)):
            n.forward(*args)
    with pytest.raises((ValueError, TypeError)):
        n.backward(x.bfloat16(), x, x, x, stats)
    with pytest.raises((ValueError, TypeError)):
        n.backward(x, x, x, x, stats[:2])
    with pytest.raises(ValueError):
        libks.ResidualNorm(16).backward(x, x, x, x, stats)
    with pytest.raises(libks.KSError):
        libks.ResidualNorm(8200, torch.ones(8200, device=DEV)).forward(torch.zeros(1, 8200, device=DEV))
