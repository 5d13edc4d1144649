"""Refusals of the residual norm, the distillation loss and beam search, without
a GPU: every argument error is found on the host before any HIP call."""
import ctypes

import pytest

from kronecker_sparse_structured_amd import libks

P = {k: (i + 1) << 36 for i, k in enumerate(
    ["x", "y", "z", "h", "gate", "stats", "pw", "pb", "qw", "qb", "s", "dz", "dh", "dx", "dy", "g0", "g1", "g2", "g3",
     "g4", "dgate", "ws", "labels", "ids", "top", "loss", "tokens", "d", "scores", "done", "lengths", "oscores",
     "otokens", "oparents", "odone", "olengths"])}
F32, BF16 = libks.ELEM_F32, libks.ELEM_BF16


# ---------------------------------------------------------------- norms

def norm_struct(width=16, kind=0, eps=1e-6, residual=1.0, elem=F32, types=(F32, F32, F32, F32), **kw):
    v = {"pw": P["pw"], "pb": P["pb"], "qw": P["qw"], "qb": P["qb"], "s": P["s"], **kw}
    return libks.ks_residual_norm_t(v["pw"], v["pb"], v["qw"], v["qb"], v["s"], width, eps, residual, kind, elem, *types)


def forward(n=None, rows=8, groups=4, **kw):
    v = {**P, **kw}
    return libks.load().ks_residual_norm(n or norm_struct(), v["x"], v["y"], v["gate"], groups, v["z"], v["h"],
                                         v["stats"], rows, None)


def test_norm_refusals():
    assert forward(norm_struct(width=0)) == libks.KS_ERR_INVALID
    assert forward(norm_struct(width=8193)) == libks.KS_ERR_UNSUPPORTED
    assert forward(norm_struct(kind=2)) == libks.KS_ERR_INVALID
    for bad in (0.0, -1.0, float("nan"), float("inf"), 1e-60):
        assert forward(norm_struct(eps=bad)) == libks.KS_ERR_INVALID
    assert forward(norm_struct(residual=float("nan"))) == libks.KS_ERR_INVALID
    assert forward(norm_struct(elem=2)) == libks.KS_ERR_DTYPE
    for k in range(4):
        types = [F32] * 4
        types[k] = 7
        assert forward(norm_struct(types=types)) == libks.KS_ERR_DTYPE
    assert forward(rows=-1) == libks.KS_ERR_BATCH and forward(rows=1 << 31) == libks.KS_ERR_BATCH
    assert forward(groups=3) == libks.KS_ERR_INVALID and forward(groups=-1) == libks.KS_ERR_INVALID
    assert forward(norm_struct(pw=None), h=None) == libks.KS_ERR_INVALID        # a bias without its weight
    assert forward(norm_struct(qw=None)) == libks.KS_ERR_INVALID
    assert forward(norm_struct(pw=None, pb=None)) == libks.KS_ERR_INVALID       # h without a norm
    assert forward(h=None) == libks.KS_ERR_INVALID
    assert forward(gate=None) == libks.KS_ERR_INVALID and forward(groups=0) == libks.KS_ERR_INVALID
    assert forward(y=None) == libks.KS_ERR_INVALID                              # z and gate without y
    assert forward(x=None) == libks.KS_ERR_NULL and forward(z=None) == libks.KS_ERR_NULL
    assert forward(norm_struct(pw=P["pw"] + 2)) == libks.KS_ERR_ALIGN
    assert forward(x=P["x"] + 2) == libks.KS_ERR_ALIGN and forward(stats=P["stats"] + 4) == libks.KS_ERR_ALIGN
    assert forward(z=P["x"] + 4) == libks.KS_ERR_OVERLAP and forward(z=P["y"]) == libks.KS_ERR_OVERLAP
    assert forward(h=P["x"]) == libks.KS_ERR_OVERLAP and forward(h=P["z"] + 8 * 64 - 4) == libks.KS_ERR_OVERLAP
    assert forward(stats=P["gate"]) == libks.KS_ERR_OVERLAP and forward(h=P["s"]) == libks.KS_ERR_OVERLAP
    assert libks.load().ks_residual_norm(None, 1, 1, 1, 0, 1, 1, 1, 1, None) == libks.KS_ERR_NULL
    assert forward(rows=0, x=None, y=None, gate=None, groups=0, z=None, h=None, stats=None) == libks.KS_OK


def grads(**kw):
    v = {"g%d" % i: P["g%d" % i] for i in range(5)}
    v.update(kw)
    return libks.ks_residual_norm_grads_t(*[v["g%d" % i] for i in range(5)])


def backward(n=None, rows=8, groups=4, g=None, ws_bytes=1 << 30, **kw):
    v = {**P, **kw}
    return libks.load().ks_residual_norm_backward(n or norm_struct(), v["dz"], v["dh"], v["x"], v["y"], v["gate"], groups,
                                                  v["stats"], v["dx"], v["dy"], g or grads(), v["dgate"], rows, v["ws"],
                                                  ws_bytes, None)


def test_norm_backward_refusals():
    size = ctypes.c_size_t(0)
    lib = libks.load()
    assert lib.ks_residual_norm_backward_workspace_size(norm_struct(), 8, 4, None) == libks.KS_ERR_NULL
    assert lib.ks_residual_norm_backward_workspace_size(norm_struct(), 8, 3, size) == libks.KS_ERR_INVALID
    assert lib.ks_residual_norm_backward_workspace_size(norm_struct(), 0, 0, size) == libks.KS_OK and size.value == 0
    assert lib.ks_residual_norm_backward_workspace_size(norm_struct(), 8, 4, size) == libks.KS_OK and size.value > 0
    assert backward(ws_bytes=size.value - 1) == libks.KS_ERR_WORKSPACE and backward(ws=None) == libks.KS_ERR_WORKSPACE
    assert backward(norm_struct(pw=None, pb=None), dh=None) == libks.KS_ERR_INVALID    # a gradient of no vector
    assert backward(norm_struct(pw=None, pb=None), g=grads(g0=None, g1=None)) == libks.KS_ERR_INVALID    # dh without h
    assert backward(groups=0, gate=None) == libks.KS_ERR_INVALID                       # a gradient of no gate
    assert backward(dy=None) == libks.KS_ERR_INVALID and backward(y=None, dy=None) == libks.KS_ERR_INVALID
    assert backward(x=None) == libks.KS_ERR_NULL and backward(dx=None) == libks.KS_ERR_NULL
    assert backward(stats=None) == libks.KS_ERR_NULL
    assert backward(ws=P["ws"] + 4) == libks.KS_ERR_ALIGN and backward(dx=P["dx"] + 1) == libks.KS_ERR_ALIGN
    assert backward(g=grads(g2=P["g2"] + 2)) == libks.KS_ERR_ALIGN
    assert backward(dx=P["dz"]) == libks.KS_ERR_OVERLAP and backward(dy=P["y"]) == libks.KS_ERR_OVERLAP
    assert backward(g=grads(g1=P["g0"])) == libks.KS_ERR_OVERLAP and backward(dgate=P["gate"]) == libks.KS_ERR_OVERLAP
    assert backward(ws=P["x"]) == libks.KS_ERR_OVERLAP and backward(g=grads(g4=P["s"])) == libks.KS_ERR_OVERLAP


# ---------------------------------------------------------------- distillation

def logits(S=2, T=3, V=10, elem=F32, **kw):
    v = {**P, **kw}
    return libks.ks_logits_t(v["x"], v["labels"], T * V, V, T, S, T, V, elem, 0)


def teacher(K=4, T=3, id_bytes=4, elem=F32, reserved=0, rows=None, **kw):
    v = {**P, **kw}
    row = K if rows is None else rows
    return libks.ks_teacher_t(v["ids"], v["top"], T * row, row, T * row, row, K, id_bytes, elem, reserved)


def distil(x=None, t=None, weight=0.5, temperature=2.0, d_seq=30, d_row=10, **kw):
    v = {**P, **kw}
    return libks.load().ks_distil_loss(x or logits(), t or teacher(), weight, temperature, v["loss"], v["tokens"],
                                       v["stats"], v["d"], d_seq, d_row, None)


def test_distil_refusals():
    nan, inf = float("nan"), float("inf")
    for w in (-0.1, 1.1, nan):
        assert distil(weight=w) == libks.KS_ERR_INVALID
    for t in (0.0, -1.0, nan, inf, 1e-30, 1e30):
        assert distil(temperature=t) == libks.KS_ERR_INVALID
    assert distil(t=teacher(K=0)) == libks.KS_ERR_INVALID and distil(t=teacher(K=257)) == libks.KS_ERR_INVALID
    assert distil(t=teacher(id_bytes=2)) == libks.KS_ERR_INVALID and distil(t=teacher(elem=3)) == libks.KS_ERR_DTYPE
    assert distil(t=teacher(reserved=1)) == libks.KS_ERR_INVALID
    assert distil(t=teacher(rows=3)) == libks.KS_ERR_INVALID                    # rows of entries that overlap
    assert distil(t=teacher(ids=None)) == libks.KS_ERR_NULL and distil(t=teacher(top=None)) == libks.KS_ERR_NULL
    assert distil(t=teacher(ids=P["ids"] + 2)) == libks.KS_ERR_ALIGN
    assert distil(t=teacher(id_bytes=8, ids=P["ids"] + 4)) == libks.KS_ERR_ALIGN
    assert distil(x=logits(V=0)) == libks.KS_ERR_INVALID and distil(x=logits(elem=2)) == libks.KS_ERR_DTYPE
    for k in ("loss", "tokens", "stats"):
        assert distil(**{k: None}) == libks.KS_ERR_NULL and distil(**{k: P[k] + 2}) == libks.KS_ERR_ALIGN
    assert distil(d_row=9) == libks.KS_ERR_INVALID
    assert distil(d=P["x"] + 4) == libks.KS_ERR_OVERLAP and distil(d=P["ids"]) == libks.KS_ERR_OVERLAP
    assert distil(d=P["x"], d_row=11, d_seq=33) == libks.KS_ERR_OVERLAP         # in place with other strides
    assert distil(tokens=P["stats"] + 72) == libks.KS_ERR_OVERLAP               # the count behind the rows' values
    assert distil(loss=P["top"]) == libks.KS_ERR_OVERLAP
    back = libks.load().ks_distil_backward
    args = (0.5, 2.0, P["stats"], None, P["d"], 30, 10, None)
    assert back(None, teacher(), *args) == libks.KS_ERR_NULL and back(logits(), None, *args) == libks.KS_ERR_NULL
    assert back(logits(), teacher(), 2.0, *args[1:]) == libks.KS_ERR_INVALID
    assert back(logits(), teacher(), *args[:2], None, *args[3:]) == libks.KS_ERR_NULL
    assert back(logits(), teacher(), *args[:4], None, *args[5:]) == libks.KS_ERR_NULL
    assert back(logits(), teacher(), *args[:4], P["stats"], *args[5:]) == libks.KS_ERR_OVERLAP
    assert back(logits(S=0), teacher(), *args) == libks.KS_OK


# ---------------------------------------------------------------- beams

def beams(R=2, W=3, V=10, eos=1, penalty=0.5, elem=F32, beam_stride=None, request_stride=None, **kw):
    v = {**P, **kw}
    b = V if beam_stride is None else beam_stride
    return libks.ks_beams_t(v["x"], v["scores"], v["done"], v["lengths"], W * b if request_stride is None
                            else request_stride, b, R, V, eos, penalty, W, elem)


def select(x=None, out=4, ws_bytes=1 << 30, **kw):
    v = {**P, **kw}
    return libks.load().ks_beam_select(x or beams(), out, v["oscores"], v["otokens"], v["oparents"], v["odone"],
                                       v["olengths"], v["ws"], ws_bytes, None)


def test_beam_refusals():
    for bad in (dict(W=0), dict(W=65), dict(V=0), dict(V=1 << 31), dict(W=64, V=1 << 25), dict(R=-1), dict(eos=10),
                dict(penalty=-0.1), dict(penalty=float("nan")), dict(beam_stride=9), dict(request_stride=29),
                dict(eos=-1)):
        assert select(beams(**bad)) == libks.KS_ERR_INVALID, bad
    assert select(beams(eos=-1, done=None)) == libks.KS_ERR_INVALID               # done out without an eos
    assert select(out=0) == libks.KS_ERR_INVALID and select(out=65) == libks.KS_ERR_INVALID
    assert select(beams(elem=2)) == libks.KS_ERR_DTYPE
    assert select(beams(lengths=None)) == libks.KS_ERR_NULL
    assert select(beams(lengths=None, penalty=0.0)) == libks.KS_ERR_NULL and select(olengths=None) == libks.KS_ERR_NULL
    assert select(beams(x=None)) == libks.KS_ERR_NULL and select(beams(scores=None)) == libks.KS_ERR_NULL
    for k in ("oscores", "otokens", "oparents", "odone"):
        assert select(**{k: None}) == libks.KS_ERR_NULL
    assert select(otokens=P["otokens"] + 4) == libks.KS_ERR_ALIGN and select(beams(x=P["x"] + 2)) == libks.KS_ERR_ALIGN
    size = ctypes.c_size_t(0)
    assert libks.load().ks_beam_workspace_size(beams(), 4, size) == libks.KS_OK
    assert select(ws_bytes=size.value - 1) == libks.KS_ERR_WORKSPACE and select(ws=None) == libks.KS_ERR_WORKSPACE
    assert libks.load().ks_beam_workspace_size(beams(), 4, None) == libks.KS_ERR_NULL
    assert select(oscores=P["scores"]) == libks.KS_ERR_OVERLAP and select(odone=P["done"] + 5) == libks.KS_ERR_OVERLAP
    assert select(ws=P["x"]) == libks.KS_ERR_OVERLAP and select(oparents=P["otokens"] + 60) == libks.KS_ERR_OVERLAP
    assert select(beams(R=0)) == libks.KS_OK
    assert libks.load().ks_beam_select(None, 1, 1, 1, 1, 1, 1, 1, 1, None) == libks.KS_ERR_NULL


def reorder(pairs, parents=P["oparents"], R=2, W=3, out=4):
    t = (libks.ks_state_t * max(len(pairs), 1))(*pairs)
    return libks.load().ks_beam_reorder(t, len(pairs), parents, R, W, out, None)


def test_reorder_refusals():
    a, b, c = P["x"], P["y"], P["z"]
    assert reorder([]) == libks.KS_OK and reorder([(a, b, 0)]) == libks.KS_OK and reorder([(a, b, 8)], R=0) == libks.KS_OK
    for bad in (dict(W=0), dict(W=65), dict(out=0), dict(out=65), dict(R=-1), dict(R=1 << 30)):
        assert reorder([(a, b, 8)], **bad) == libks.KS_ERR_INVALID, bad
    assert reorder([(a, b, -1)]) == libks.KS_ERR_INVALID
    assert reorder([(None, b, 8)]) == libks.KS_ERR_NULL and reorder([(a, None, 8)]) == libks.KS_ERR_NULL
    assert reorder([(a, b, 8)], parents=None) == libks.KS_ERR_NULL
    assert reorder([(a, b, 8)], parents=P["ids"] + 2) == libks.KS_ERR_ALIGN
    # src has 6 rows, dst 8
    assert reorder([(a, a, 8)]) == libks.KS_ERR_OVERLAP and reorder([(a, a + 47, 8)]) == libks.KS_ERR_OVERLAP
    assert reorder([(a + 63, a, 8)]) == libks.KS_ERR_OVERLAP
    assert reorder([(a, b, 8), (c, b + 60, 8)]) == libks.KS_ERR_OVERLAP          # two results
    assert reorder([(a, b, 8), (b + 60, c, 8)]) == libks.KS_ERR_OVERLAP          # another state's source
    assert reorder([(a, b, 8)], parents=b) == libks.KS_ERR_OVERLAP
    # a large source that reaches past a smaller one in between
    assert reorder([(a, b, 1000), (a + 8, a + 5000, 8)]) == libks.KS_ERR_OVERLAP


def test_workspace_of_beams_grows_with_what_it_holds():
    def size(out, **kw):
        n = ctypes.c_size_t(0)
        assert libks.load().ks_beam_workspace_size(beams(**kw), out, n) == libks.KS_OK
        return n.value

    # 10 values: one slice, at most 10 keys of 8 bytes and two sums a beam
    assert size(4) == 6 * 40 and size(64) == 6 * 88
    assert size(4, V=50257, elem=BF16) > size(4, V=1000, elem=BF16)


@pytest.mark.parametrize("call", ["distillation_loss", "beam_select", "beam_reorder", "ResidualNorm"])
def test_host_tensors_are_refused(call):
    import torch
    x, ids = torch.zeros(2, 3, 10), torch.zeros(2, 3, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        if call == "distillation_loss":
            libks.distillation_loss(x, torch.zeros(2, 3, dtype=torch.int64), ids, torch.zeros(2, 3, 4))
        elif call == "beam_select":
            libks.beam_select(x, torch.zeros(2, 3))
        elif call == "beam_reorder":
            libks.beam_reorder([x], ids[:, :, 0].contiguous())
        else:
            libks.ResidualNorm(10, torch.ones(10))


def test_calls_run_on_their_tensors_device(monkeypatch):
    import contextlib

    import torch
    entered = []

    @contextlib.contextmanager
    def device(index):
        entered.append(index)
        yield

    monkeypatch.setattr(libks, "_current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", device)
    assert libks._on_device(0, lambda a: a + 1, 4) == 5 and entered == []
    assert libks._on_device(3, lambda a: a + 1, 4) == 5 and entered == [3]
