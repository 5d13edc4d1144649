"""Fine-tuning a Kronecker-sparse layer: the operators around its product, as cases to measure.

Three operators that a user of the layer meets next to it:

* adapter: a shared Kronecker-sparse projection with low-rank adapters of many
  requests beside it. Row n of X belongs to adapter g = ids[n] (no adapter if g
  is not in [0, G)):
      H[n] = scale[g] X[n] A[g]^T,   Y[n] = X[n] W^T + H[n] B[g]^T
  and its gradients with a frozen W:
      E[n] = scale[g] dY[n] B[g],    dX[n] = dY[n] W + E[n] A[g]
      dA[g] = sum_{n of g} E[n]^T X[n],   dB[g] = sum_{n of g} dY[n]^T H[n]
* preference: log probabilities of labelled tokens from logits, and the paired
  preference loss on them with its gradient. Sequences 0..P-1 are the chosen
  ones, P..2P-1 the rejected ones; a negative label masks its token.
      l[s,t] = x[s,t,label] - log sum_v exp x[s,t,v]
      R[s] = sum_t (l[s,t] - ref[s,t]),  z_i = beta (R[i] - R[P+i])
      loss_i = (1-e) log(1 + exp(-z_i)) + e log(1 + exp(z_i))
      dx[s,t,v] = c[s] (1[v = label] - softmax(x[s,t])_v),
      c[i] = -c[P+i] = beta (e sigma(z_i) - (1-e) sigma(-z_i)) / P
* adamw: one step over many tensors, the moments in 32 bits or in 8 with one
  scale for each 256 values and moment:
      m = b1 m + (1-b1) g,  v = b2 v + (1-b2) g^2
      p = (1 - lr wd) p - lr/(1-b1^t) m / (sqrt(v/(1-b2^t)) + eps)
  with g scaled so that the norm over all tensors is at most max_norm. In 8
  bits m is held as s k|k| / 127^2 with a signed k, v as s k^4 / 255^4; a value
  between two codes goes to the upper one with the probability that keeps its
  mean, by a random number hashed from the step's seed and the value's index.
"""
import math
import random

import torch

own = False

PAIR = "1,64,16,64;64,8,8,8"      # 1024 -> 4096, two factors
UP = "4,64,16,6"                  # 384 -> 1536, one factor
MONARCH = "32,32,32,1;1,32,32,32"  # 1024 -> 1024
ODD = "3,5,7,2"                   # 42 -> 30
BLOCK = 256                       # values that share a scale in 8 bits


def listed():
    return [
        # one token of one request: latency
        {"name": "adapter_one_token", "op": "adapter", "train": False, "patterns": PAIR, "rows": 1, "adapters": 8,
         "rank": 16, "dtype": "bf16"},
        # a decoding batch: each row a request of its own, with its adapter
        {"name": "adapter_decode", "op": "adapter", "train": False, "patterns": PAIR, "rows": 64, "adapters": 32,
         "rank": 16, "dtype": "bf16"},
        # prompts of several requests, 16 x 1024 tokens together
        {"name": "adapter_prompts", "op": "adapter", "train": False, "patterns": PAIR, "rows": 16384, "adapters": 8,
         "rank": 16, "dtype": "bf16"},
        # a training step's forward and backward, an odd number of rows
        {"name": "adapter_train", "op": "adapter", "train": True, "patterns": PAIR, "rows": 4099, "adapters": 4,
         "rank": 32, "dtype": "bf16"},
        # the same over 128 x 197 image tokens in fp32
        {"name": "adapter_train_images", "op": "adapter", "train": True, "patterns": UP, "rows": 25216, "adapters": 2,
         "rank": 8, "dtype": "f32"},
        # a few short answers over a small vocabulary: latency
        {"name": "preference_small", "op": "preference", "train": True, "pairs": 2, "tokens": 33, "vocab": 4096,
         "dtype": "f32", "smoothing": 0.0},
        # the reference model's log probabilities of a batch: no gradient
        {"name": "preference_reference", "op": "preference", "train": False, "pairs": 8, "tokens": 512,
         "vocab": 32000, "dtype": "bf16", "smoothing": 0.0},
        # a training batch over an odd vocabulary: rows that start at any even byte
        {"name": "preference_train", "op": "preference", "train": True, "pairs": 8, "tokens": 512, "vocab": 50257,
         "dtype": "bf16", "smoothing": 0.1},
        # the adapters of four layers: small tensors, latency
        {"name": "adamw_adapters", "op": "adamw", "layers": 4, "rank": 16, "table": 0, "params": "f32",
         "grads": "f32", "bits": 32, "clip": True},
        # every factor and bias of 24 layers, bf16 weights
        {"name": "adamw_layers_8bit", "op": "adamw", "layers": 24, "rank": 0, "table": 0, "params": "bf16",
         "grads": "bf16", "bits": 8, "clip": False},
        # the layers with a token table of 50257 x 1024
        {"name": "adamw_model", "op": "adamw", "layers": 24, "rank": 0, "table": 51463168, "params": "f32",
         "grads": "f32", "bits": 32, "clip": True},
        {"name": "adamw_model_8bit", "op": "adamw", "layers": 24, "rank": 0, "table": 51463168, "params": "f32",
         "grads": "bf16", "bits": 8, "clip": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adapter", "preference", "adamw"])
    if op == "adapter":
        train = rng.random() < 0.5
        return {"op": op, "train": train, "patterns": rng.choice([PAIR, UP, MONARCH, ODD]),
                "rows": _log(rng, 1, 4099 if train else 16384), "adapters": _log(rng, 1, 32),
                "rank": rng.choice([4, 5, 8, 13, 16, 24, 32]), "dtype": rng.choice(["bf16", "f32"])}
    if op == "preference":
        vocab = _log(rng, 50, 50257)
        tokens = _log(rng, 1, 512)
        pairs = max(1, min(_log(rng, 1, 16), 8 * 512 * 50257 // (2 * tokens * vocab)))
        return {"op": op, "train": rng.random() < 0.7, "pairs": pairs, "tokens": tokens, "vocab": vocab,
                "dtype": rng.choice(["bf16", "f32"]), "smoothing": rng.choice([0.0, 0.1])}
    bits = rng.choice([32, 8])
    return {"op": op, "layers": _log(rng, 1, 24), "rank": rng.choice([0, 5, 8, 16]),
            "table": rng.choice([0, _log(rng, 1000, 40000000)]), "params": rng.choice(["bf16", "f32"]),
            "grads": rng.choice(["bf16", "f32"]), "bits": bits, "clip": bits == 32 and rng.random() < 0.5}


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _patterns(text):
    return [tuple(int(v) for v in p.split(",")) for p in text.split(";")]


def _widths(patterns):
    a, b, c, d = patterns[0]
    e, f, g, h = patterns[-1]
    return a * c * d, e * f * h


def _adapter_ids(case, seed):
    """The adapter of each row: up to 64 rows each their own request; more rows: requests of ragged
    length one after another, one of them without an adapter."""
    r = random.Random(seed * 7919 + 13)
    n, count = case["rows"], case["adapters"]
    if n <= 64:
        return [r.randrange(-1, count) if n > 1 else r.randrange(count) for _ in range(n)]
    cuts = sorted(r.randrange(n + 1) for _ in range(2 * count))
    ids, at = [], 0
    for k, end in enumerate(cuts + [n]):
        ids += [-1 if k == count else r.randrange(count)] * (end - at)
        at = end
    return ids


def _sizes(case):
    """Elements of each tensor of an optimizer step."""
    sizes = []
    for _ in range(case["layers"]):
        if case["rank"]:
            sizes += [case["rank"] * 1024, case["rank"] * 4096]     # adapters of a 1024 -> 4096 layer
        else:
            sizes += [65536, 32768, 4096, 1023]                     # its factors, a bias, an odd vector
    return sizes + ([case["table"]] if case["table"] else [])


HYPER = {"lr": 1e-3, "b1": 0.9, "b2": 0.999, "eps": 1e-8, "wd": 0.01, "step": 20, "max_norm": 1.0}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    s = {"case": case}
    if case["op"] == "adapter":
        t = _type(case["dtype"])
        ps = _patterns(case["patterns"])
        n_in, n_out = _widths(ps)
        n, count, rank = case["rows"], case["adapters"], case["rank"]
        s["X"] = normal(n, n_in).to(t)
        s["W"] = [(normal(a, d, b, c) / math.sqrt(c)).to(t) for a, b, c, d in ps]
        s["A"] = (normal(count, rank, n_in) / math.sqrt(n_in)).to(t)
        s["B"] = (normal(count, n_out, rank) / math.sqrt(rank)).to(t)
        s["scale"] = 0.5 + torch.rand(count, generator=gen, device="cuda")
        s["ids"] = torch.tensor(_adapter_ids(case, seed), dtype=torch.int32).cuda()
        if case["train"]:
            s["dY"] = normal(n, n_out)
        s["patterns"] = ps
        if own:  # the layer's handle on its weights, which a program keeps
            from kronecker_sparse_structured_amd import libks
            s["layer"] = libks.AdapterChain(s["W"], ps, s["A"], s["B"], s["scale"])
    elif case["op"] == "preference":
        P, T, V = case["pairs"], case["tokens"], case["vocab"]
        x = normal(2 * P, T, V)
        x *= 2
        label = torch.randint(V, (2 * P, T), generator=gen, device="cuda")
        # trained models put their labels some way up
        x.scatter_add_(2, label[:, :, None], (4 * torch.rand((2 * P, T, 1), generator=gen, device="cuda")))
        s["logits"] = x.to(_type(case["dtype"]))
        at = torch.gather(s["logits"], 2, label[:, :, None])[:, :, 0].float()
        del x
        # a prompt in front, padding behind: masked
        r = random.Random(seed * 104729 + 5)
        lo = torch.tensor([r.randrange(T // 4 + 1) for _ in range(2 * P)]).cuda()
        hi = torch.tensor([T - r.randrange(T // 4 + 1) for _ in range(2 * P)]).cuda()
        pos = torch.arange(T, device="cuda")[None, :]
        s["labels"] = torch.where((pos >= lo[:, None]) & (pos < hi[:, None]), label, torch.full_like(label, -100))
        # the reference model is near the policy: log sum exp of N(0, 4) logits is near log V + 2
        s["ref"] = at - (math.log(V) + 2) + 0.3 * normal(2 * P, T)
    else:
        sizes = _sizes(case)
        starts = [0]
        for n in sizes:
            starts.append(starts[-1] + -(-n // BLOCK) * BLOCK)
        total = starts[-1]
        live = torch.zeros(total, device="cuda")
        for n, a in zip(sizes, starts):
            live[a:a + n] = 1.0

        def views(flat):
            return [flat[a:a + n] for n, a in zip(sizes, starts)]

        # gradients and states of a run under way: sizes differ from block to block
        level = torch.exp(normal(total // BLOCK)).repeat_interleave(BLOCK)
        s["p"] = (0.1 * normal(total) * live).to(_type(case["params"]))
        s["g"] = (0.01 * level * normal(total) * live).to(_type(case["grads"]))
        if case["bits"] == 32:
            s["m"] = 0.003 * level * normal(total) * live
            s["v"] = (0.01 * level * (0.2 + torch.rand(total, generator=gen, device="cuda"))).square() * 0.02 * live
            s["scales"] = None
        else:
            s["m"] = (torch.randint(-127, 128, (total,), generator=gen, device="cuda") * live).to(torch.int8)
            s["v"] = (torch.randint(40, 256, (total,), generator=gen, device="cuda") * live).to(torch.uint8)
            per = level[::BLOCK]
            s["scales"] = torch.stack([0.009 * per, (0.012 * per).square() * 0.02], dim=1).contiguous()
        s["seed"] = (seed * 2654435761) % (1 << 32)
        if own:  # the optimizer, which a program keeps with its parameters, gradient buffers and states
            from kronecker_sparse_structured_amd import libks
            scales = None
            if case["bits"] == 8:
                scales = [s["scales"][a // BLOCK:a // BLOCK + -(-n // BLOCK)] for n, a in zip(sizes, starts)]
            s["steps"] = libks.AdamW(views(s["p"]), views(s["g"]), views(s["m"]), views(s["v"]), scales)
            if case["bits"] == 8:
                s["wide"] = torch.zeros(total, device="cuda"), torch.zeros(total, device="cuda")
                s["wide_views"] = views(s["wide"][0]), views(s["wide"][1])
    return s


def run(s):
    return {"adapter": _adapter, "preference": _preference, "adamw": _adamw}[s["case"]["op"]](s)


# ---------------------------------------------------------------- adapters

def _factor(x, w, p):
    """x W^T of one factor in 32 bits: (n, a c d) -> (n, a b d)."""
    a, b, c, d = p
    xs = x.view(-1, a, c, d).permute(1, 3, 0, 2).reshape(a * d, -1, c).contiguous()
    ws = w.reshape(a * d, b, c).transpose(1, 2).contiguous()
    return torch.bmm(xs, ws).view(a, d, -1, b).permute(2, 0, 3, 1).reshape(-1, a * b * d)


def _factor_dx(dy, w, p):
    a, b, c, d = p
    ds = dy.view(-1, a, b, d).permute(1, 3, 0, 2).reshape(a * d, -1, b).contiguous()
    return torch.bmm(ds, w.reshape(a * d, b, c).contiguous()).view(a, d, -1, c).permute(2, 0, 3, 1).reshape(-1, a * c * d)


def _fold(f, x, pairs):
    """f applied with each (weights, pattern) in turn."""
    return x if not pairs else _fold(f, f(x, *pairs[0]), pairs[1:])


def _adapter(s):
    train = s["case"]["train"]
    if own:
        layer = s["layer"]
        if not train:
            return layer.matmul(s["X"], s["ids"])
        Y, H = layer.matmul(s["X"], s["ids"], keep=True)
        dX, dA, dB = layer.backward(s["dY"], s["X"], H, s["ids"])
        return {"Y": Y, "dX": dX, "dA": dA, "dB": dB}
    X, A, B = s["X"].float(), s["A"].float(), s["B"].float()
    W = list(zip(map(torch.Tensor.float, s["W"]), s["patterns"]))
    count, rank, n_in = A.shape
    # every adapter's product, kept where it is the row's own
    mine = (s["ids"][:, None] == torch.arange(count, device=X.device)[None, :]).float() * s["scale"][None, :]
    mine = mine.repeat_interleave(rank, dim=1)
    A = A.reshape(count * rank, n_in)
    B = B.permute(0, 2, 1).reshape(count * rank, -1)
    H = (X @ A.t()) * mine
    Y = _fold(_factor, X, W) + H @ B
    if not train:
        return Y
    dY = s["dY"]
    E = (dY @ B.t()) * mine
    dX = _fold(_factor_dx, dY, W[::-1]) + E @ A
    dA = (E.t() @ X).view(count, rank, n_in)
    dB = (H.t() @ dY).view(count, rank, -1).permute(0, 2, 1).contiguous()
    return {"Y": Y, "dX": dX, "dA": dA, "dB": dB}


def _adapter_exact(case, s):
    X = s["X"].double()
    n_in, n_out = _widths(s["patterns"])

    def dense(w, p):
        a, b, c, d = p
        out = torch.zeros(a * b * d, a * c * d, dtype=torch.float64, device=w.device)
        i = torch.arange(a * d * b * c, device=w.device)
        ga, be, de, al = i % c, i // c % b, i // (c * b) % d, i // (c * b * d)
        out[(al * b + be) * d + de, (al * c + ga) * d + de] = w.double().reshape(-1)
        return out

    W = [dense(w, p) for w, p in zip(s["W"], s["patterns"])]
    Y = X
    for w in W:
        Y = Y @ w.t()
    rows = [(s["ids"] == g).nonzero()[:, 0] for g in range(case["adapters"])]
    H = {}
    for g, at in enumerate(rows):
        H[g] = float(s["scale"][g]) * (X[at] @ s["A"][g].double().t())
        Y[at] += H[g] @ s["B"][g].double().t()
    if not case["train"]:
        return Y
    dY = s["dY"].double()
    dX = dY
    for w in reversed(W):
        dX = dX @ w
    dA = torch.zeros(s["A"].shape, dtype=torch.float64, device=X.device)
    dB = torch.zeros(s["B"].shape, dtype=torch.float64, device=X.device)
    for g, at in enumerate(rows):
        E = float(s["scale"][g]) * (dY[at] @ s["B"][g].double())
        dX[at] += E @ s["A"][g].double()
        dA[g] = E.t() @ X[at]
        dB[g] = dY[at].t() @ H[g]
    return {"Y": Y, "dX": dX, "dA": dA, "dB": dB}


# ---------------------------------------------------------------- preferences

BETA = 0.1


def _preference(s):
    case = s["case"]
    if own:
        from kronecker_sparse_structured_amd import libks
        if not case["train"]:
            total, tokens = libks.sequence_logp(s["logits"], s["labels"])
            return {"logp": total, "tokens": tokens}
        loss, rewards, tokens, dlogits = libks.preference_loss(s["logits"], s["labels"], s["ref"], beta=BETA,
                                                               smoothing=case["smoothing"])
        return {"loss": loss, "rewards": rewards, "tokens": tokens, "dlogits": dlogits}
    x = s["logits"].float()
    on = s["labels"] >= 0
    at = s["labels"].clamp(min=0)[:, :, None]
    x = x - x.amax(dim=2, keepdim=True)
    e = x.exp()
    total = e.sum(dim=2, keepdim=True)
    tokens = torch.where(on, (torch.gather(x, 2, at) - total.log())[:, :, 0], 0.0)
    if not case["train"]:
        return {"logp": tokens.sum(dim=1), "tokens": tokens}
    P, smooth = case["pairs"], case["smoothing"]
    rewards = BETA * torch.where(on, tokens - s["ref"], 0.0).sum(dim=1)
    z = rewards[:P] - rewards[P:]
    down = (-z.abs()).exp()
    more = torch.log1p(down)
    loss = ((1 - smooth) * (more + (-z).clamp(min=0)) + smooth * (more + z.clamp(min=0))).mean()
    up = torch.where(z >= 0, 1.0, down) / (1 + down)          # sigma(z)
    un = torch.where(z >= 0, down, 1.0) / (1 + down)          # sigma(-z)
    c = BETA * (smooth * up - (1 - smooth) * un) / P
    c = torch.cat([c, -c])[:, None] * on
    d = e * (-c[:, :, None] / total)
    d.scatter_add_(2, at, c[:, :, None])
    return {"loss": loss, "rewards": rewards, "tokens": tokens, "dlogits": d.to(s["logits"].dtype)}


def _preference_exact(case, s):
    S, T, V = s["logits"].shape
    P, e = case["pairs"], case["smoothing"]
    tokens = torch.zeros(S, T, dtype=torch.float64, device="cuda")
    on = s["labels"] >= 0
    for q in range(S):
        x = s["logits"][q].double()
        l = torch.logsumexp(x, dim=1)
        t = on[q].nonzero()[:, 0]
        tokens[q, t] = x[t, s["labels"][q, t]] - l[t]
    if not case["train"]:
        return {"logp": tokens.sum(dim=1), "tokens": tokens}
    ratio = (tokens - s["ref"].double()) * on
    rewards = BETA * ratio.sum(dim=1)
    z = rewards[:P] - rewards[P:]
    loss = ((1 - e) * torch.nn.functional.softplus(-z) + e * torch.nn.functional.softplus(z)).mean()
    slope = BETA * (e * torch.sigmoid(z) - (1 - e) * torch.sigmoid(-z)) / P
    d = torch.zeros(S, T, V, dtype=torch.float64, device="cuda")
    for q in range(S):
        t = on[q].nonzero()[:, 0]
        row = -torch.softmax(s["logits"][q, t].double(), dim=1)
        row[torch.arange(len(t), device="cuda"), s["labels"][q, t]] += 1
        d[q, t] = row * (slope[q] if q < P else -slope[q - P])
    return {"loss": loss, "rewards": rewards, "tokens": tokens, "dlogits": d}


# ---------------------------------------------------------------- AdamW

def _random(total, seed, device, salt=0):
    """32 random bits for each index: a multiplicative hash of it and the seed."""
    M = 0xFFFFFFFF
    x = (torch.arange(total, device=device, dtype=torch.int64) * 0x9E3779B1 + seed) & M
    x = x ^ salt
    x = x ^ (x >> 16)
    x = (x * 0xAADDE6A9) & M
    x = x ^ (x >> 15)
    x = (x * 0xBEDE544D) & M
    return x ^ (x >> 16)


def _m_of(k, scale):
    k = k.float().view(-1, BLOCK)
    return (k * k.abs() * (scale / 16129.0)).view(-1)


def _v_of(k, scale):
    k = k.float().view(-1, BLOCK)
    return (((k * k) * (k * k)) * (scale / 4228250625.0)).view(-1)


def _m_codes(m, chance):
    m = m.view(-1, BLOCK)
    size = m.abs()
    scale = size.amax(dim=1, keepdim=True).clamp(min=1e-30)
    u = size * (16129.0 / scale)
    k = u.sqrt().floor().clamp(max=127)
    k = torch.where(k * k > u, k - 1, k)
    step = 2 * k + 1
    k = k + (chance.view(-1, BLOCK) * step < u - k * k)
    return (k.clamp(max=127) * m.sign()).view(-1).to(torch.int8), scale


def _v_codes(v, chance):
    v = v.view(-1, BLOCK)
    scale = v.amax(dim=1, keepdim=True).clamp(min=1e-28)
    u = v * (4228250625.0 / scale)
    k = u.sqrt().sqrt().floor().clamp(max=255)
    low = (k * k) * (k * k)
    k = torch.where(low > u, k - 1, k)
    low = (k * k) * (k * k)
    high = ((k + 1) * (k + 1)) * ((k + 1) * (k + 1))
    k = k + (chance.view(-1, BLOCK) * (high - low) < u - low)
    k = torch.where((k < 1) & (v > 0), 1.0, k)
    return k.clamp(max=255).view(-1).to(torch.uint8), scale


def _adamw(s):
    case, h = s["case"], HYPER
    if own:
        s["steps"].step(step=h["step"], lr=h["lr"], betas=(h["b1"], h["b2"]), eps=h["eps"], weight_decay=h["wd"],
                        max_norm=h["max_norm"] if case["clip"] else None, seed=s["seed"])
        if case["bits"] == 32:
            return {"p": s["p"], "m": s["m"], "v": s["v"]}
        s["steps"].state_values(*s["wide_views"])
        return {"p": s["p"], "m": s["wide"][0], "v": s["wide"][1]}
    p, g = s["p"].float(), s["g"].float()
    if case["clip"]:
        norm = (g * g).sum().sqrt()
        g = g * (h["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    wide = case["bits"] == 32
    m = s["m"] if wide else _m_of(s["m"], s["scales"][:, :1])
    v = s["v"] if wide else _v_of(s["v"], s["scales"][:, 1:])
    m = m * h["b1"] + g * (1 - h["b1"])
    v = v * h["b2"] + (g * g) * (1 - h["b2"])
    root = v.sqrt() * (1 / math.sqrt(1 - h["b2"] ** h["step"])) + h["eps"]
    p = p * (1 - h["lr"] * h["wd"]) - (m / root) * (h["lr"] / (1 - h["b1"] ** h["step"]))
    s["p"].copy_(p)
    if wide:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return {"p": s["p"], "m": s["m"], "v": s["v"]}
    bits = _random(p.numel(), s["seed"], p.device)
    mk, ms = _m_codes(m, (bits & 0xFFFF).float() / 65536)
    vk, vs = _v_codes(v, (bits >> 16).float() / 65536)
    s["m"].copy_(mk)
    s["v"].copy_(vk)
    s["scales"].copy_(torch.cat([ms, vs], dim=1))
    return {"p": s["p"], "m": _m_of(mk, ms), "v": _v_of(vk, vs)}


def _adamw_exact(case, s):
    h = HYPER
    p, g = s["p"].double(), s["g"].double()
    if case["clip"]:
        g = g * min(1.0, h["max_norm"] / (float(g.norm()) + 1e-6))
    m, v = s["m"].double(), s["v"].double()
    if case["bits"] == 8:
        wide = s["scales"].double().repeat_interleave(BLOCK, dim=0)
        m, v = wide[:, 0] * m * m.abs() / 127 ** 2, wide[:, 1] * (v / 255) ** 4
    m = h["b1"] * m + (1 - h["b1"]) * g
    v = h["b2"] * v + (1 - h["b2"]) * g ** 2
    mhat, vhat = m / (1 - h["b1"] ** h["step"]), v / (1 - h["b2"] ** h["step"])
    p = p - h["lr"] * h["wd"] * p - h["lr"] * mhat / (vhat.sqrt() + h["eps"])
    if case["bits"] == 8:
        # a value between two codes: the upper one if its place between them is above the random number
        bits = _random(p.numel(), s["seed"], p.device)

        def held(x, levels, power, least, chance, floor):
            x = x.view(-1, BLOCK)
            top = x.amax(dim=1, keepdim=True).clamp(min=least)
            u = x / top * levels ** power
            k = (u ** (1 / power) + 1e-12).floor().clamp(max=levels)
            up = chance.view(-1, BLOCK) * ((k + 1) ** power - k ** power) < u - k ** power
            k = (k + up).clamp(max=levels)
            if floor:
                k = torch.where((k < 1) & (x > 0), 1.0, k)
            return (top * (k / levels) ** power).view(-1)

        m = m.sign() * held(m.abs(), 127, 2, 1e-30, (bits & 0xFFFF) / 65536.0, False)
        v = held(v, 255, 4, 1e-28, (bits >> 16) / 65536.0, True)
    return {"p": p, "m": m, "v": v}


def exact(case, seed):
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    return {"adapter": _adapter_exact, "preference": _preference_exact, "adamw": _adamw_exact}[case["op"]](case, s)


def work(case):
    if case["op"] == "adapter":
        ps = _patterns(case["patterns"])
        n_in, n_out = _widths(ps)
        n, rank, size = case["rows"], case["rank"], 2 if case["dtype"] == "bf16" else 4
        used = min(case["adapters"], n)
        weights = sum(a * b * c * d for a, b, c, d in ps) + used * rank * (n_in + n_out)
        base = sum(2 * n * a * b * c * d for a, b, c, d in ps)
        low = 2 * n * rank * (n_in + n_out)
        moved = n * (n_in * size + n_out * 4 + 4) + weights * size
        if not case["train"]:
            return {"bytes": moved, "flops": base + low}
        moved += n * (n_out + n_in) * 4 + case["adapters"] * rank * (n_in + n_out) * 4
        return {"bytes": moved, "flops": 2 * base + 3 * low}
    if case["op"] == "preference":
        rows, size = 2 * case["pairs"] * case["tokens"], 2 if case["dtype"] == "bf16" else 4
        moved = rows * (case["vocab"] * size + 8 + 4)
        if not case["train"]:
            return {"bytes": moved, "flops": 4 * rows * case["vocab"]}
        return {"bytes": moved + rows * (case["vocab"] * size + 4), "flops": 7 * rows * case["vocab"]}
    n = sum(_sizes(case))
    size = {"f32": 4, "bf16": 2}
    state = 16 if case["bits"] == 32 else 4 + 8 + 16 / BLOCK   # in 8 bits: codes read and written, values returned
    return {"bytes": n * (size[case["grads"]] + 2 * size[case["params"]] + state), "flops": 15 * n}
