"""Refusals of the operators around the product, without a GPU: every argument
error is found on the host before any HIP call."""
import ctypes

import pytest

from kronecker_sparse_structured_amd import libks

P = dict(A=0x10000000, B=0x20000000, scale=0x30000000, ids=0x38000000, X=0x40000000, Y=0x50000000, H=0x60000000,
         dY=0x70000000, dX=0x80000000, dA=0x90000000, dB=0xA0000000, ws=0xB0000000)
F32, BF16, BF16W = libks.DTYPE_F32, libks.DTYPE_BF16, libks.DTYPE_BF16W


def adapters(n_in=16, n_out=24, rank=4, count=3, **kw):
    v = {**P, **kw}
    return libks.ks_adapters_t(v["A"], v["B"], v["scale"], n_in, n_out, rank, count)


def forward(ad=None, batch=8, dt=F32, ws_bytes=1 << 30, **kw):
    v = {**P, **kw}
    return libks.load().ks_adapter_matmul(ad if ad is not None else adapters(), v["ids"], v["X"], v["Y"], v["H"], batch,
                                          dt, v["ws"], ws_bytes, None)


def test_adapter_refusals():
    assert forward(batch=-1) == libks.KS_ERR_BATCH and forward(batch=1 << 31) == libks.KS_ERR_BATCH
    assert forward(dt=7) == libks.KS_ERR_DTYPE
    for bad in (dict(rank=0), dict(rank=libks.load() and 257), dict(count=0), dict(count=65536), dict(n_in=0),
                dict(n_out=1 << 31), dict(n_in=1 << 30, rank=4)):
        assert forward(adapters(**bad)) == libks.KS_ERR_INVALID, bad
    assert forward(adapters(rank=256), batch=1 << 23) == libks.KS_ERR_INVALID
    for k in ("A", "B", "scale"):
        assert forward(adapters(**{k: None})) == libks.KS_ERR_NULL
    for k in ("ids", "X", "Y", "H"):
        assert forward(**{k: None}) == libks.KS_ERR_NULL
    assert forward(X=P["X"] + 2) == libks.KS_ERR_ALIGN and forward(Y=P["Y"] + 1) == libks.KS_ERR_ALIGN
    assert forward(adapters(A=P["A"] + 1), dt=BF16) == libks.KS_ERR_ALIGN
    assert forward(Y=P["X"] + 8 * 16 * 4 - 4) == libks.KS_ERR_OVERLAP
    assert forward(H=P["Y"] + 4) == libks.KS_ERR_OVERLAP
    assert forward(Y=P["ids"]) == libks.KS_ERR_OVERLAP
    assert libks.load().ks_adapter_matmul(None, P["ids"], P["X"], P["Y"], P["H"], 8, F32, None, 0,
                                          None) == libks.KS_ERR_NULL
    size = ctypes.c_size_t(0)
    assert libks.load().ks_adapter_workspace_size(adapters(), 1000, size) == libks.KS_OK and size.value >= 4000
    assert forward(batch=1000, ws_bytes=size.value - 1) == libks.KS_ERR_WORKSPACE
    assert forward(batch=1000, ws=P["ws"] + 4) == libks.KS_ERR_ALIGN
    assert forward(batch=1000, ws=P["X"]) == libks.KS_ERR_OVERLAP
    assert forward(batch=0, X=None, Y=None, ids=None, H=None) == libks.KS_OK


def backward(ad=None, batch=8, dt=F32, ws_bytes=1 << 30, **kw):
    v = {**P, **kw}
    return libks.load().ks_adapter_backward(ad if ad is not None else adapters(), v["ids"], v["dY"], v["X"], v["H"],
                                            v["dX"], v["dA"], v["dB"], batch, dt, v["ws"], ws_bytes, None)


def test_adapter_backward_refusals():
    size = ctypes.c_size_t(0)
    assert libks.load().ks_adapter_backward_workspace_size(adapters(), 8, size) == libks.KS_OK and size.value > 0
    assert libks.load().ks_adapter_backward_workspace_size(adapters(), 8, None) == libks.KS_ERR_NULL
    assert backward(ws_bytes=size.value - 1) == libks.KS_ERR_WORKSPACE and backward(ws=None) == libks.KS_ERR_WORKSPACE
    assert backward(ws=P["ws"] + 8) == libks.KS_ERR_ALIGN
    assert backward(dA=None) == libks.KS_ERR_NULL and backward(dY=None) == libks.KS_ERR_NULL
    assert backward(H=None) == libks.KS_ERR_NULL and backward(ids=None) == libks.KS_ERR_NULL
    assert backward(dX=P["dY"]) == libks.KS_ERR_OVERLAP and backward(dA=P["dB"]) == libks.KS_ERR_OVERLAP
    assert backward(ws=P["X"]) == libks.KS_ERR_OVERLAP
    assert backward(dt=-1) == libks.KS_ERR_DTYPE
    assert backward(batch=0, dA=None, dB=None) == libks.KS_OK


PS = [(1, 4, 4, 4), (4, 6, 4, 1)]      # 16 -> 16 -> 24
WP = (ctypes.c_void_p * 2)(0xC0000000, 0xD0000000)


def chain(ps=PS, ad=None, n=2, batch=8, dt=F32, ws_bytes=1 << 30, w=WP, **kw):
    v = {**P, **kw}
    return libks.load().ks_chain_adapter_matmul(libks._patterns(ps), n, w, ad if ad is not None else adapters(), v["ids"],
                                                v["X"], v["Y"], v["H"], batch, dt, v["ws"], ws_bytes, None)


def test_chain_refusals():
    size = ctypes.c_size_t(0)
    pats = libks._patterns(PS)
    assert libks.load().ks_chain_adapter_workspace_size(pats, 2, adapters(), 2000, F32, size) == libks.KS_OK
    assert size.value >= 2000 * 4 * 4                    # H, where the caller keeps none
    assert chain(batch=2000, ws_bytes=size.value - 1) == libks.KS_ERR_WORKSPACE
    assert chain(ad=adapters(n_in=20)) == libks.KS_ERR_CHAIN_MISMATCH
    assert chain(n=1) == libks.KS_ERR_CHAIN_MISMATCH
    assert chain(ps=[(1, 4, 0, 4), (4, 6, 4, 1)]) == libks.KS_ERR_PATTERN
    assert chain(w=(ctypes.c_void_p * 2)(0xC0000000, None)) == libks.KS_ERR_NULL
    assert chain(batch=2000, ws=P["X"]) == libks.KS_ERR_OVERLAP
    assert chain(dt=9) == libks.KS_ERR_DTYPE and chain(batch=-4) == libks.KS_ERR_BATCH
    assert chain(batch=0, X=None) == libks.KS_OK
    lib = libks.load()

    def back(ws_bytes=1 << 30, w=WP, dx=P["dX"], wt=None, **kw):
        v = {**P, **kw}
        return lib.ks_chain_adapter_backward(pats, 2, w, wt, adapters(), v["ids"], v["dY"], v["X"], v["H"], dx, v["dA"],
                                             v["dB"], 8, F32, v["ws"], ws_bytes, None)

    assert lib.ks_chain_adapter_backward_workspace_size(pats, 2, adapters(), 8, F32, 0, size) == libks.KS_OK
    assert back(ws_bytes=size.value - 1) == libks.KS_ERR_WORKSPACE
    assert back(dx=None) == libks.KS_ERR_NULL and back(w=None) == libks.KS_ERR_NULL
    assert back(dx=0xC0000000) == libks.KS_ERR_OVERLAP and back(dB=None) == libks.KS_ERR_NULL
    assert back(wt=0xE0000008) == libks.KS_ERR_ALIGN and back(wt=P["dX"]) == libks.KS_ERR_OVERLAP
    less = ctypes.c_size_t(0)
    assert lib.ks_chain_adapter_backward_workspace_size(pats, 2, adapters(), 8, F32, 1, less) == libks.KS_OK
    assert less.value <= size.value
    assert lib.ks_chain_transpose_size(pats, 2, F32, less) == libks.KS_OK and less.value >= (64 + 96) * 4
    assert lib.ks_chain_transpose_size(pats, 2, 5, less) == libks.KS_ERR_DTYPE
    assert lib.ks_chain_transpose(pats, 2, WP, None, F32, None) == libks.KS_ERR_NULL
    assert lib.ks_chain_transpose(pats, 2, WP, 0xE0000004, F32, None) == libks.KS_ERR_ALIGN
    assert lib.ks_chain_transpose(pats, 2, WP, 0xC0000000, F32, None) == libks.KS_ERR_OVERLAP
    assert lib.ks_chain_transpose(pats, 2, (ctypes.c_void_p * 2)(None, 16), 0xE0000000, F32, None) == libks.KS_ERR_NULL


def test_weights_of_the_chain_apart_from_everything_written():
    size = ctypes.c_size_t(0)
    pats = libks._patterns(PS)
    lib = libks.load()
    assert lib.ks_chain_adapter_workspace_size(pats, 2, adapters(), 2000, F32, size) == libks.KS_OK
    at = lambda a: (ctypes.c_void_p * 2)(a, WP[1])
    assert chain(w=at(P["H"])) == libks.KS_ERR_OVERLAP
    assert chain(batch=2000, w=at(P["ws"] + size.value - 16)) == libks.KS_ERR_OVERLAP
    for name in ("dA", "dB"):
        assert lib.ks_chain_adapter_backward(pats, 2, at(P[name]), None, adapters(), P["ids"], P["dY"], P["X"], P["H"],
                                             P["dX"], P["dA"], P["dB"], 8, F32, P["ws"], 1 << 30, None) == \
            libks.KS_ERR_OVERLAP


def logits(**kw):
    v = dict(data=0x10000000, labels=0x20000000, seq_stride=40, row_stride=10, label_stride=4, sequences=2, tokens=4,
             vocab=10, elem=libks.ELEM_F32, reserved=0)
    v.update(kw)
    return libks.ks_logits_t(*[v[n] for n, _ in libks.ks_logits_t._fields_])


def logp(x, tokens=0x30000000, total=0x40000000, stats=0x50000000):
    return libks.load().ks_sequence_logp(x, tokens, total, stats, None)


def loss(x=None, ref=0x30000000, ref_stride=4, beta=0.1, e=0.0, out=0x40000000, rewards=0x41000000, tokens=0x42000000,
         grad=0x43000000, stats=0x44000000, d=None, d_seq=0, d_row=0):
    return libks.load().ks_preference_loss(x if x is not None else logits(), ref, ref_stride, beta, e, out, rewards, tokens,
                                           grad, stats, d, d_seq, d_row, None)


def test_preference_refusals():
    for bad in (dict(vocab=0), dict(sequences=-1), dict(tokens=-1), dict(row_stride=9), dict(seq_stride=39),
                dict(label_stride=3), dict(reserved=1), dict(sequences=1 << 31), dict(tokens=1 << 30, sequences=4)):
        assert logp(logits(**bad)) == libks.KS_ERR_INVALID, bad
    assert logp(logits(elem=2)) == libks.KS_ERR_DTYPE
    assert logp(logits(data=None)) == libks.KS_ERR_NULL and logp(logits(labels=None)) == libks.KS_ERR_NULL
    assert logp(logits(), tokens=None) == libks.KS_ERR_NULL and logp(logits(), total=None) == libks.KS_ERR_NULL
    assert logp(logits(data=0x10000002)) == libks.KS_ERR_ALIGN and logp(logits(labels=0x20000004)) == libks.KS_ERR_ALIGN
    assert logp(logits(), tokens=0x10000000) == libks.KS_ERR_OVERLAP
    assert logp(logits(), total=0x30000004) == libks.KS_ERR_OVERLAP
    assert logp(logits(sequences=0)) == libks.KS_OK
    assert libks.load().ks_sequence_logp(None, 1, 1, None, None) == libks.KS_ERR_NULL
    assert loss(logits(sequences=3)) == libks.KS_ERR_INVALID
    for kw in (dict(beta=0.0), dict(beta=float("nan")), dict(e=-0.1), dict(e=1.5), dict(ref_stride=3),
               dict(d=0x60000000, d_seq=40, d_row=9), dict(d=0x60000000, d_seq=30, d_row=10)):
        assert loss(**kw) == libks.KS_ERR_INVALID, kw
    for kw in (dict(ref=None), dict(out=None), dict(rewards=None), dict(tokens=None), dict(grad=None), dict(stats=None)):
        assert loss(**kw) == libks.KS_ERR_NULL, kw
    assert loss(stats=0x42000000) == libks.KS_ERR_OVERLAP and loss(rewards=0x10000000) == libks.KS_ERR_OVERLAP
    # the gradient may replace the logits, but not sit across them
    assert loss(d=0x10000004, d_seq=40, d_row=10) == libks.KS_ERR_OVERLAP
    assert loss(d=0x10000000, d_seq=60, d_row=15) == libks.KS_ERR_OVERLAP
    lib = libks.load()
    assert lib.ks_preference_backward(logits(), None, 8, None, 16, 40, 10, None) == libks.KS_ERR_NULL
    assert lib.ks_preference_backward(logits(), 0x50000000, 0x51000000, None, 0x60000001, 40, 10, None) == libks.KS_ERR_ALIGN
    assert lib.ks_preference_backward(logits(), 0x50000000, 0x51000000, None, 0x50000000, 40, 10, None) == libks.KS_ERR_OVERLAP


def tensor(**kw):
    v = dict(p=0x10000000, g=0x20000000, m=0x30000000, v=0x40000000, scales=0x50000000, n=100, p_elem=0, g_elem=0)
    v.update(kw)
    return (libks.ks_adamw_tensor_t * 1)(libks.ks_adamw_tensor_t(*[v[n] for n, _ in libks.ks_adamw_tensor_t._fields_]))


def step(t, n=1, norm=None, **kw):
    v = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0, max_norm=0.0, step=1, seed=0, state_bits=32)
    v.update(kw)
    o = libks.ks_adamw_options_t(*[v[n_] for n_, _ in libks.ks_adamw_options_t._fields_])
    return libks.load().ks_adamw_step(t, n, o, norm, None)


def test_adamw_refusals():
    for kw in (dict(step=0), dict(state_bits=16), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1.0),
               dict(lr=float("inf")), dict(max_norm=-1.0), dict(max_norm=float("nan"))):
        assert step(tensor(), **kw) == libks.KS_ERR_INVALID, kw
    assert step(tensor(), max_norm=1.0) == libks.KS_ERR_NULL
    assert step(tensor(n=-1)) == libks.KS_ERR_INVALID and step(tensor(n=1 << 31)) == libks.KS_ERR_INVALID
    assert step(tensor(g_elem=5)) == libks.KS_ERR_DTYPE and step(tensor(p_elem=5)) == libks.KS_ERR_DTYPE
    for k in ("p", "g", "m", "v"):
        assert step(tensor(**{k: None})) == libks.KS_ERR_NULL
    assert step(tensor(scales=None), state_bits=8) == libks.KS_ERR_NULL
    assert step(tensor(m=0x30000002)) == libks.KS_ERR_ALIGN and step(tensor(p=0x10000001, p_elem=1)) == libks.KS_ERR_ALIGN
    assert step(tensor(g=0x10000004)) == libks.KS_ERR_OVERLAP and step(tensor(v=0x30000000)) == libks.KS_ERR_OVERLAP
    assert step(tensor(scales=0x30000000), state_bits=8) == libks.KS_ERR_OVERLAP
    assert step(None) == libks.KS_ERR_NULL and step(None, n=0) == libks.KS_OK and step(tensor(n=0, p=None)) == libks.KS_OK
    lib = libks.load()
    size = ctypes.c_size_t(0)
    assert lib.ks_grad_norm_workspace_size(tensor(n=1 << 20), 1, size) == libks.KS_OK
    assert lib.ks_grad_norm(tensor(n=1 << 20), 1, 0x60000000, 0x70000000, size.value - 1, None) == libks.KS_ERR_WORKSPACE
    assert lib.ks_grad_norm(tensor(), 1, None, 0x70000000, 1 << 20, None) == libks.KS_ERR_NULL
    assert lib.ks_grad_norm(tensor(g=None), 1, 0x60000000, 0x70000000, 1 << 20, None) == libks.KS_ERR_NULL
    assert lib.ks_grad_norm(tensor(), 1, 0x20000000, 0x70000000, 1 << 20, None) == libks.KS_ERR_OVERLAP
    outs = (ctypes.c_void_p * 1)(0x60000000), (ctypes.c_void_p * 1)(0x30000000)
    assert lib.ks_adamw_state_values(tensor(), 1, *outs, None) == libks.KS_ERR_OVERLAP
    assert lib.ks_adamw_state_values(tensor(), 1, None, outs[0], None) == libks.KS_ERR_NULL
    assert lib.ks_adamw_state_values(tensor(v=None), 1, outs[0], outs[1], None) == libks.KS_ERR_NULL


@pytest.mark.parametrize("name", ["ks_adapters_t", "ks_logits_t", "ks_adamw_tensor_t", "ks_adamw_options_t"])
def test_structures_have_no_hidden_padding(name):
    t = getattr(libks, name)
    assert ctypes.sizeof(t) == sum(ctypes.sizeof(f) for _, f in t._fields_)
