"""A stack of Kronecker-sparse layers around its products, as cases to measure.

Three operators that a user meets who puts such layers in place of a model's
dense ones: the norms, gate and residual between the layers, the loss against
the dense model, and the choice of the next tokens.

* norm: what stands between two blocks. The block's output y is normed, gated,
  scaled and added to the residual x; the sum is normed for the next block.
      u = post(y),  z = x + a s u g,  h = pre(z)
  norms over the last dimension, by root mean square, or by mean and variance:
      rms(v) = v / sqrt(mean v^2 + eps) w,  layer(v) = (v - mean v) / sqrt(var v + eps) w + b
  s is a vector, a a number, and row n's gate is g[n / (rows / groups)]. The
  gradients are of x, y, the gate and every vector, from those of z and of h.
* distil: the loss of logits against a teacher's K highest logits of each token
  (id < 0: fewer than K), mixed with the labels' (label < 0: masked token).
      q = softmax(top / tau) over the K,  p = softmax(x / tau),  p1 = softmax(x)
      token = w tau^2 sum_k q_k (log q_k - log p[id_k]) - (1 - w) log p1[label]
      loss = sum of tokens / N,  N tokens are not masked
      dx_v = (w tau (p_v - q_v) + (1 - w) (p1_v - 1[v = label])) / N
* beam: the best continuations of each request's beams, and their states.
      candidate (b, v): score[b] + x[b, v] - log sum exp x[b]; of a finished
      beam only (b, eos), at its own score
  ranked by score / length^penalty, the lowest b V + v first among equals. Row j
  of every state becomes the row of the beam that candidate j continues.
"""
import math
import random

import torch

own = False


def listed():
    return [
        # one token through the end of a block: latency
        {"name": "norm_token", "op": "norm", "train": False, "rows": 1, "width": 1024, "kind": "rms", "post": True,
         "groups": 0, "scale": True, "x": "bf16", "y": "f32", "h": "bf16", "params": "bf16"},
        # prompts of 16 x 1024 tokens, the 1024-wide layers of a language model; no norm after the block
        {"name": "norm_prompts", "op": "norm", "train": False, "rows": 16384, "width": 1024, "kind": "layer",
         "post": False, "groups": 0, "scale": False, "x": "f32", "y": "f32", "h": "bf16", "params": "f32"},
        # a training step of 128 images of 197 tokens, each image with its gate
        {"name": "norm_train_images", "op": "norm", "train": True, "rows": 25216, "width": 384, "kind": "layer",
         "post": True, "groups": 128, "scale": True, "x": "f32", "y": "f32", "h": "f32", "params": "f32"},
        # a training step over an odd number of tokens, each with its gate
        {"name": "norm_train", "op": "norm", "train": True, "rows": 4099, "width": 1024, "kind": "rms", "post": True,
         "groups": 4099, "scale": True, "x": "bf16", "y": "f32", "h": "bf16", "params": "f32"},
        # the same over wide rows, no gate
        {"name": "norm_train_wide", "op": "norm", "train": True, "rows": 4096, "width": 4096, "kind": "rms",
         "post": True, "groups": 0, "scale": True, "x": "bf16", "y": "bf16", "h": "bf16", "params": "f32"},
        # a few short answers over a small vocabulary: latency
        {"name": "distil_small", "op": "distil", "train": True, "sequences": 4, "tokens": 33, "vocab": 4096, "top": 16,
         "weight": 0.5, "tau": 2.0, "dtype": "f32"},
        # how far a held-out batch is from its teacher: no gradient
        {"name": "distil_held_out", "op": "distil", "train": False, "sequences": 8, "tokens": 512, "vocab": 32000,
         "top": 32, "weight": 1.0, "tau": 1.0, "dtype": "f32"},
        # a training batch over an odd vocabulary: rows that start at any even byte
        {"name": "distil_train", "op": "distil", "train": True, "sequences": 16, "tokens": 512, "vocab": 50257,
         "top": 64, "weight": 0.9, "tau": 2.0, "dtype": "bf16"},
        # one request: latency
        {"name": "beam_one", "op": "beam", "requests": 1, "beams": 4, "vocab": 50257, "dtype": "bf16", "penalty": 0.0,
         "history": 64, "cache": 0},
        # a batch of requests, some of their beams finished
        {"name": "beam_batch", "op": "beam", "requests": 64, "beams": 4, "vocab": 50257, "dtype": "bf16",
         "penalty": 0.6, "history": 512, "cache": 0},
        # many beams over fp32 logits
        {"name": "beam_many", "op": "beam", "requests": 32, "beams": 16, "vocab": 32000, "dtype": "f32",
         "penalty": 1.0, "history": 128, "cache": 0},
        # the beams' caches follow them: 2 MB a beam
        {"name": "beam_caches", "op": "beam", "requests": 16, "beams": 4, "vocab": 4096, "dtype": "f32",
         "penalty": 0.0, "history": 128, "cache": 1048576},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "distil", "beam"])
    if op == "norm":
        width = rng.choice([384, 1024, 4096, _log(rng, 8, 8192)])
        rows = max(1, min(_log(rng, 1, 25216), 25216 * 384 // width))
        count = rng.choice([0, 0, 1, rows, _log(rng, 1, rows)])
        if count:
            rows = rows // count * count        # whole groups
        return {"op": op, "train": rng.random() < 0.6, "rows": rows, "width": width,
                "kind": rng.choice(["rms", "layer"]), "post": rng.random() < 0.6, "groups": count,
                "scale": rng.random() < 0.6, "x": rng.choice(["bf16", "f32"]), "y": rng.choice(["bf16", "f32"]),
                "h": rng.choice(["bf16", "f32"]), "params": rng.choice(["bf16", "f32"])}
    if op == "distil":
        vocab, tokens = _log(rng, 50, 50257), _log(rng, 1, 512)
        sequences = max(1, min(_log(rng, 1, 32), 8 * 512 * 50257 // (tokens * vocab)))
        return {"op": op, "train": rng.random() < 0.7, "sequences": sequences, "tokens": tokens, "vocab": vocab,
                "top": min(vocab, _log(rng, 1, 128)), "weight": rng.choice([1.0, 0.9, 0.5]),
                "tau": rng.choice([1.0, 2.0]), "dtype": rng.choice(["bf16", "f32"])}
    beams = _log(rng, 1, 16)
    return {"op": op, "requests": max(1, min(_log(rng, 1, 64), 512 // beams)), "beams": beams,
            "vocab": _log(rng, 50, 50257), "dtype": rng.choice(["bf16", "f32"]),
            "penalty": rng.choice([0.0, 0.6, 1.0]), "history": _log(rng, 1, 512),
            "cache": rng.choice([0, _log(rng, 100, 200000)])}


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


EPS = 1e-5
RESIDUAL = 0.5
EOS = 2


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda", dtype=torch.float32)

    s = {"case": case}
    if case["op"] == "norm":
        n, d, params = case["rows"], case["width"], _type(case["params"])
        # a residual that has grown over the layers, with an offset; the block's output is smaller
        s["x"] = (2 * normal(n, d) + 0.5 * normal(d)).to(_type(case["x"]))
        s["y"] = ((0.5 + uniform(n, 1)) * normal(n, d) + 0.2).to(_type(case["y"]))
        s["gate"] = (1 + 0.3 * normal(case["groups"], d)).to(_type(case["y"])) if case["groups"] else None
        s["dz"] = normal(n, d).to(_type(case["x"])) if case["train"] else None
        s["dh"] = normal(n, d).to(_type(case["h"])) if case["train"] else None
        layer = case["kind"] == "layer"
        vector = {"pre_weight": True, "pre_bias": layer, "post_weight": case["post"],
                  "post_bias": case["post"] and layer, "scale": case["scale"]}
        s["vectors"] = {k: ((0.0 if "bias" in k else 1.0) + 0.2 * normal(d)).to(params) if on else None
                        for k, on in vector.items()}
        if own:  # the norm's handle on its vectors, which a program keeps
            from kronecker_sparse_structured_amd import libks
            s["norm"] = libks.ResidualNorm(d, **s["vectors"], kind=case["kind"], eps=EPS, residual=RESIDUAL)
    elif case["op"] == "distil":
        S, T, V, K = case["sequences"], case["tokens"], case["vocab"], case["top"]
        x = normal(S, T, V)
        # the teacher's logits: near the student's, and higher on what it is sure of
        at = torch.randint(V, (S, T, 4), generator=gen, device="cuda")
        x.scatter_add_(2, at, 8 * uniform(S, T, 4))
        s["top"], s["ids"] = (x + 0.5 * normal(S, T, V)).topk(K, dim=2)
        s["ids"] = s["ids"].to(torch.int32)
        s["top"] = s["top"].to(_type(case["dtype"]))
        # some rows were cut off at a share of the probability: fewer than K
        some = torch.randint(1, K + 1, (S, T, 1), generator=gen, device="cuda")
        cut = (torch.arange(K, device="cuda") >= some) & (uniform(S, T, 1) < 0.3)
        s["ids"] = torch.where(cut, torch.full_like(s["ids"], -1), s["ids"])
        s["logits"] = x.to(_type(case["dtype"]))
        label = torch.where(uniform(S, T) < 0.7, s["ids"][:, :, 0].long(),
                            torch.randint(V, (S, T), generator=gen, device="cuda"))
        del x
        # a prompt in front, padding behind: masked
        r = random.Random(seed * 104729 + 5)
        lo = torch.tensor([r.randrange(T // 4 + 1) for _ in range(S)]).cuda()
        hi = torch.tensor([T - r.randrange(T // 4 + 1) for _ in range(S)]).cuda()
        pos = torch.arange(T, device="cuda")[None, :]
        s["labels"] = torch.where((pos >= lo[:, None]) & (pos < hi[:, None]), label, torch.full_like(label, -100))
    else:
        B, W, V = case["requests"], case["beams"], case["vocab"]
        x = 2 * normal(B, W, V)
        # a few likely tokens each
        x.scatter_add_(2, torch.randint(V, (B, W, 6), generator=gen, device="cuda"), 9 * uniform(B, W, 6))
        s["logits"] = x.to(_type(case["dtype"]))
        del x
        s["lengths"] = torch.randint(4, 40, (B, 1), generator=gen, device="cuda", dtype=torch.int32).repeat(1, W)
        s["scores"] = -2.0 * s["lengths"] - 4 * uniform(B, W)
        # some beams have ended, earlier than the others; every eighth request has just begun, with one beam
        s["done"] = uniform(B, W) < 0.15
        s["lengths"] = torch.where(s["done"], (s["lengths"] + 1) // 2, s["lengths"])
        begun = (torch.arange(B, device="cuda") % 8 == 7)[:, None]
        s["done"] &= ~begun
        s["lengths"] = torch.where(begun, torch.zeros_like(s["lengths"]), s["lengths"])
        first = torch.full((1, W), -math.inf, device="cuda")
        first[0, 0] = 0.0
        s["scores"] = torch.where(begun, first, s["scores"])
        s["states"] = [torch.randint(V, (B, W, case["history"]), generator=gen, device="cuda", dtype=torch.int32)]
        if case["cache"]:
            s["states"].append(normal(B, W, case["cache"]).to(torch.bfloat16))
        s["spare"] = [torch.empty_like(t) for t in s["states"]]    # where a program keeps the next step's
    return s


def run(s):
    return {"norm": _norm, "distil": _distil, "beam": _beam}[s["case"]["op"]](s)


# ---------------------------------------------------------------- norms

def _normed(v, layer):
    """(v normed, 1 / its deviation) in v's type."""
    if layer:
        v = v - v.mean(dim=1, keepdim=True)
    r = (v.square().mean(dim=1, keepdim=True) + EPS).rsqrt()
    return v * r, r


def _norm_back(d, n, r, layer):
    """The gradient behind a norm, from that of its normed values n."""
    out = d - n * (d * n).mean(dim=1, keepdim=True)
    if layer:
        out = out - d.mean(dim=1, keepdim=True)
    return out * r


def _norm(s):
    case = s["case"]
    if own:
        norm = s["norm"]
        if not case["train"]:
            z, h = norm.forward(s["x"], s["y"], s["gate"], dtype=_type(case["h"]))
            return {"z": z, "h": h}
        z, h, stats = norm.forward(s["x"], s["y"], s["gate"], dtype=_type(case["h"]), keep=True)
        g = norm.backward(s["dz"], s["dh"], s["x"], s["y"], stats, s["gate"])
        return {"z": z, "h": h, **{k: v for k, v in g._asdict().items() if v is not None}}
    return _norm_plain(s, torch.float32)


def _norm_plain(s, wide):
    """The formulas in `wide` bits, rounded to the outputs' types if those are 32."""
    case, layer = s["case"], s["case"]["kind"] == "layer"
    v = {k: None if t is None else t.to(wide) for k, t in s["vectors"].items()}
    x, y = s["x"].to(wide), s["y"].to(wide)
    n, d = x.shape

    def rounded(t, like):
        return t.to(like) if wide == torch.float32 else t

    ones = torch.ones((), dtype=wide, device=x.device)
    u = y
    if case["post"]:
        yn, yr = _normed(y, layer)
        u = yn * v["post_weight"]
        if layer:
            u = u + v["post_bias"]
    scale = v["scale"] if case["scale"] else ones
    gate = s["gate"].to(wide).repeat_interleave(n // case["groups"], dim=0) if case["groups"] else ones
    z = x + RESIDUAL * scale * gate * u
    zn, zr = _normed(z, layer)
    h = zn * v["pre_weight"]
    if layer:
        h = h + v["pre_bias"]
    out = {"z": rounded(z, s["x"].dtype), "h": rounded(h, _type(case["h"]))}
    if not case["train"]:
        return out
    dz, dh = s["dz"].to(wide), s["dh"].to(wide)
    dx = dz + _norm_back(dh * v["pre_weight"], zn, zr, layer)
    du = RESIDUAL * scale * gate * dx
    dy = _norm_back(du * v["post_weight"], yn, yr, layer) if case["post"] else du
    out["dx"], out["dy"] = rounded(dx, s["x"].dtype), rounded(dy, s["y"].dtype)
    out["pre_weight"] = (dh * zn).sum(dim=0)
    if layer:
        out["pre_bias"] = dh.sum(dim=0)
    if case["post"]:
        out["post_weight"] = (du * yn).sum(dim=0)
        if layer:
            out["post_bias"] = du.sum(dim=0)
    if case["scale"]:
        out["scale"] = (RESIDUAL * dx * u * gate).sum(dim=0)
    if case["groups"]:
        dg = (RESIDUAL * dx * u * scale).view(case["groups"], -1, d).sum(dim=1)
        out["gate"] = rounded(dg, s["gate"].dtype)
    return out


def _norm_exact(case, s):
    """From the definitions in 64 bits; the gradients by differentiating them."""
    layer, d = case["kind"] == "layer", case["width"]
    leaf = {k: t.double().requires_grad_(case["train"]) for k, t in
            {"x": s["x"], "y": s["y"], "gate": s["gate"], **s["vectors"]}.items() if t is not None}

    def norm(v, w, b):
        if layer:
            return torch.nn.functional.layer_norm(v, (d,), w, b, EPS)
        return v / torch.sqrt(torch.mean(v * v, dim=-1, keepdim=True) + EPS) * w

    u = norm(leaf["y"], leaf["post_weight"], leaf.get("post_bias")) if case["post"] else leaf["y"]
    if case["scale"]:
        u = u * leaf["scale"]
    if case["groups"]:
        u = (u.view(case["groups"], -1, d) * leaf["gate"][:, None, :]).reshape(-1, d)
    z = leaf["x"] + RESIDUAL * u
    h = norm(z, leaf["pre_weight"], leaf.get("pre_bias"))
    out = {"z": z.detach(), "h": h.detach()}
    if case["train"]:
        grads = torch.autograd.grad((z, h), list(leaf.values()), (s["dz"].double(), s["dh"].double()))
        g = dict(zip(leaf, grads))
        out.update(dx=g.pop("x"), dy=g.pop("y"), **g)
    return out


# ---------------------------------------------------------------- distillation

def _distil(s):
    case = s["case"]
    if own:
        from kronecker_sparse_structured_amd import libks
        loss, tokens, d = libks.distillation_loss(s["logits"], s["labels"], s["ids"], s["top"], weight=case["weight"],
                                                  temperature=case["tau"], grad=case["train"])
        return {"loss": loss, "tokens": tokens, "dlogits": d} if case["train"] else {"loss": loss, "tokens": tokens}
    w, tau = case["weight"], case["tau"]
    x = s["logits"].float()
    on = s["labels"] >= 0
    count = on.sum().clamp(min=1).float()
    x = x - x.amax(dim=2, keepdim=True)
    have = s["ids"] >= 0
    at = s["ids"].clamp(min=0).long()
    t = torch.where(have, s["top"].float() * (1 / tau), -math.inf)
    t = t - t.amax(dim=2, keepdim=True)
    total = t.exp().sum(dim=2, keepdim=True)
    q = t.exp() / total
    e = (x * (1 / tau)).exp() if tau != 1 else x.exp()
    sums = e.sum(dim=2, keepdim=True)
    logp = torch.gather(x, 2, at) * (1 / tau) - sums.log()
    tokens = w * tau * tau * torch.where(have, q * (t - total.log() - logp), 0.0).sum(dim=2)
    place = s["labels"].clamp(min=0)[:, :, None]
    if w < 1:
        e1 = x.exp() if tau != 1 else e
        sums1 = e1.sum(dim=2, keepdim=True)
        tokens = tokens - (1 - w) * (torch.gather(x, 2, place) - sums1.log())[:, :, 0]
    tokens = torch.where(on, tokens, 0.0)
    out = {"loss": tokens.sum() / count, "tokens": tokens}
    if not case["train"]:
        return out
    c = (on / count)[:, :, None]
    d = e * (w * tau * c / sums)
    if w < 1:
        d += e1 * ((1 - w) * c / sums1)
        d.scatter_add_(2, place, -(1 - w) * c)
    d.scatter_add_(2, at, torch.where(have, -w * tau * c * q, 0.0))
    out["dlogits"] = d.to(s["logits"].dtype)
    return out


def _distil_exact(case, s):
    S, T, V = s["logits"].shape
    w, tau = case["weight"], case["tau"]
    on = s["labels"] >= 0
    count = max(1, int(on.sum()))
    tokens = torch.zeros(S, T, dtype=torch.float64, device="cuda")
    d = torch.zeros(S, T, V, dtype=torch.float64, device="cuda") if case["train"] else None
    for i in range(S):
        r = on[i].nonzero()[:, 0]
        if not len(r):
            continue
        x, ids, label = s["logits"][i, r].double(), s["ids"][i, r].long(), s["labels"][i, r]
        top = s["top"][i, r].double().masked_fill(ids < 0, -math.inf)
        logq = torch.log_softmax(top / tau, dim=1)
        logp = torch.log_softmax(x / tau, dim=1)
        q = logq.exp()
        part = q * (logq - logp.gather(1, ids.clamp(min=0)))
        value = w * tau ** 2 * part.masked_fill(ids < 0, 0.0).sum(dim=1)
        plain = torch.log_softmax(x, dim=1)
        value = value - (1 - w) * plain.gather(1, label[:, None])[:, 0]
        tokens[i, r] = value
        if case["train"]:
            g = w * tau * logp.exp() + (1 - w) * plain.exp()
            g.scatter_add_(1, ids.clamp(min=0), -w * tau * q.masked_fill(ids < 0, 0.0))
            g[torch.arange(len(r), device="cuda"), label] -= 1 - w
            d[i, r] = g / count
    out = {"loss": tokens.sum() / count, "tokens": tokens}
    return {**out, "dlogits": d} if case["train"] else out


# ---------------------------------------------------------------- beams

def _beam(s):
    case = s["case"]
    if own:
        from kronecker_sparse_structured_amd import libks
        b = libks.beam_select(s["logits"], s["scores"], done=s["done"], lengths=s["lengths"], eos=EOS,
                              length_penalty=case["penalty"])
        states = libks.beam_reorder(s["states"], b.parents, out=s["spare"])
        return {**b._asdict(), "states": states}
    x = s["logits"].float() + 0.0                      # -0 is 0
    B, W, V = x.shape
    K = min(W, V)
    # a beam's best: by value, then by the lowest token; 64 bits from here on, since ranks of two
    # beams' candidates may lie close together
    bits = x.view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * 2 ** 32 + (V - 1 - torch.arange(V, device=x.device))
    at = V - 1 - (key.topk(K, dim=2)[0] & 0xFFFFFFFF)
    wide = x.double()
    top = wide.amax(dim=2, keepdim=True)
    value = torch.gather(wide, 2, at) - top - (wide - top).exp().sum(dim=2, keepdim=True).log()
    # a finished beam goes on as it is
    done = s["done"][:, :, None]
    first = torch.arange(K, device=x.device) == 0
    value = s["scores"].double()[:, :, None] + torch.where(done, torch.where(first, 0.0, -math.inf), value)
    token = torch.where(done, torch.full_like(at, EOS), at)
    length = s["lengths"][:, :, None] + (~done).int()
    rank = value / length.clamp(min=1).double() ** case["penalty"]
    # best first, the lowest beam and token first among equals
    order = torch.argsort((torch.arange(W, device=x.device)[:, None] * V + token).view(B, W * K), dim=1)
    order = order.gather(1, torch.sort(rank.view(B, W * K).gather(1, order), dim=1, descending=True, stable=True)[1])
    order = order[:, :W]
    parents = order // K
    scores = value.view(B, W * K).gather(1, order)
    dead = scores == -math.inf
    parents = torch.where(dead, 0, parents)
    tokens = torch.where(dead, EOS, token.view(B, W * K).gather(1, order))
    lengths = torch.where(dead, 0, length.expand(B, W, K).reshape(B, W * K).gather(1, order))
    rows = (torch.arange(B, device=x.device)[:, None] * W + parents).view(-1)
    return {"scores": scores.float(), "tokens": tokens, "parents": parents.int(),
            "done": (tokens == EOS) | dead, "lengths": lengths,
            "states": [t.view(B * W, -1).index_select(0, rows).view(t.shape) for t in s["states"]]}


def _beam_exact(case, s):
    B, W, V = s["logits"].shape
    out = {"scores": torch.full((B, W), -math.inf, dtype=torch.float64, device="cuda"),
           "tokens": torch.full((B, W), EOS, device="cuda"),
           "parents": torch.zeros(B, W, dtype=torch.int32, device="cuda"),
           "done": torch.ones(B, W, dtype=torch.bool, device="cuda"),
           "lengths": torch.zeros(B, W, dtype=torch.int32, device="cuda")}
    for b in range(B):
        value = s["scores"][b].double()[:, None] + torch.log_softmax(s["logits"][b].double(), dim=1)
        for w in s["done"][b].nonzero()[:, 0].tolist():
            value[w] = -math.inf
            value[w, EOS] = s["scores"][b, w].double()
        length = s["lengths"][b] + (~s["done"][b]).int()
        rank = (value / length.clamp(min=1).double()[:, None] ** case["penalty"]).view(-1)
        order = torch.sort(rank, descending=True, stable=True)[1][:W]
        order = order[rank[order] > -math.inf]
        n, parent = len(order), order // V
        out["scores"][b, :n] = value.view(-1)[order]
        out["tokens"][b, :n] = order % V
        out["parents"][b, :n] = parent.int()
        out["done"][b, :n] = order % V == EOS
        out["lengths"][b, :n] = length[parent]
    pick = out["parents"].long()
    out["states"] = [torch.stack([t[b][pick[b]] for b in range(B)]) for t in s["states"]]
    return out


def exact(case, seed):
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    return {"norm": _norm_exact, "distil": _distil_exact, "beam": _beam_exact}[case["op"]](case, s)


def work(case):
    size = {"f32": 4, "bf16": 2}
    if case["op"] == "norm":
        n = case["rows"] * case["width"]
        x, y, h, p = (size[case[k]] for k in ("x", "y", "h", "params"))
        layer = case["kind"] == "layer"
        vectors = (1 + layer) * (1 + case["post"]) + case["scale"]
        gates = case["groups"] * case["width"] * y
        moved = n * (2 * x + y + h) + case["width"] * vectors * p + gates
        if not case["train"]:
            return {"bytes": moved, "flops": 12 * n}
        return {"bytes": moved + n * (2 * x + y + h) + case["width"] * vectors * 4 + gates, "flops": 40 * n}
    if case["op"] == "distil":
        rows = case["sequences"] * case["tokens"]
        each = size[case["dtype"]]
        moved = rows * (case["vocab"] * each + case["top"] * (4 + each) + 8 + 4)
        if not case["train"]:
            return {"bytes": moved, "flops": 6 * rows * case["vocab"]}
        return {"bytes": moved + rows * case["vocab"] * each, "flops": 10 * rows * case["vocab"]}
    beams = case["requests"] * case["beams"]
    states = case["history"] * 4 + case["cache"] * 2
    return {"bytes": beams * (case["vocab"] * size[case["dtype"]] + 2 * states + 9 + 21),
            "flops": 5 * beams * case["vocab"]}
