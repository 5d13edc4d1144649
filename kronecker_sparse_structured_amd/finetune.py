"""Preference fine-tuning of adapters beside a frozen KS layer, end to end on
synthetic data.

    python -m kronecker_sparse_structured_amd.finetune [--steps 60] [--state-bits 8]
        [--blocks 2] [--distil-steps 40] [--beams 4]

The model is a table of token vectors and one AdapterLinear whose KS factors map
1024 -> 4096; its outputs are the logits of 4096 tokens. There are several
tasks, each with its own adapter: task g wants token t to be followed by a token
of its own. A batch holds pairs of answers of all tasks, the chosen one (the
task's successors) and the rejected one (random tokens); the reference model is
the same layer with the adapters left out (ids -1). Each step runs the adapters
forward and backward, the preference loss with its gradient, and AdamW over the
adapters. At the end one token of each of many requests is decoded in one call,
every row with the adapter of its request.

With --blocks the token vectors first go through that many KS layers 1024 -> 1024
with norms and residuals around them. With --distil-steps the layers are trained
before that, against a dense model's 64 highest logits (and the tokens it would
choose). With --beams the requests are also answered by a beam search of several
tokens.
"""
from __future__ import annotations

import argparse

from . import layer, libks, optim

PATTERNS = [(1, 64, 16, 64), (64, 8, 8, 8)]   # 1024 -> 4096
BLOCK = [(32, 32, 32, 1), (1, 32, 32, 32)]    # 1024 -> 1024
TOP = 64                                      # logits of the dense model that are kept


def distil(base, body, table, steps, lr, state_bits, seed, report=None, tokens=32, weight=0.9, temperature=2.0):
    """Trains the layers (and the blocks in front of them) against a dense
    model's highest logits; returns the losses."""
    import torch
    device, out = table.device, []
    gen = torch.Generator(device=device).manual_seed(seed + 2)
    dense = torch.randn(base.n_out, base.n_in, generator=gen, device=device) * (3 / base.n_in ** 0.5)
    params = [*base.parameters(), *(body.parameters() if body is not None else ())]
    opt = optim.AdamW(params, lr=lr, weight_decay=0.0, state_bits=state_bits, max_norm=1.0, seed=seed)
    for _ in range(steps):
        x = table[torch.randint(len(table), (16, tokens), generator=gen, device=device)]
        with torch.no_grad():
            top, ids = (x.float() @ dense.t()).topk(TOP, dim=2)
        labels = ids[:, :, 0].contiguous()
        labels[:, 0] = -100
        opt.zero_grad()
        h = x if body is None else body(x)
        loss, _ = layer.distillation_loss(base(h), labels, ids, top, weight, temperature)
        loss.backward()
        opt.step()
        out.append(float(loss.detach()))
        if report:
            report(len(out), out[-1], None)
    return out


def search(logits_of, first, beams, steps):
    """Beam search: first (R,) tokens, logits_of(tokens (R, W)) -> (R, W, V). Returns
    the tokens (R, beams, steps) and scores (R, beams), best first."""
    import torch
    scores = torch.zeros(len(first), 1, device=first.device)
    tokens, history = first[:, None], None
    for _ in range(steps):
        best = libks.beam_select(logits_of(tokens), scores, beams)
        scores, tokens = best.scores, best.tokens
        if history is not None:
            history, = libks.beam_reorder([history], best.parents)
        last = tokens[:, :, None]
        history = last if history is None else torch.cat([history, last], dim=2)
    return history, scores


def run(steps=60, tasks=4, pairs=8, tokens=32, rank=16, state_bits=8, lr=5e-3, beta=0.1, seed=0, device="cuda",
        report=None, blocks=0, distil_steps=0, beams=0, answer=3):
    """Trains and returns {"loss": [...], "margin": [...], "correct": share of
    greedily decoded tokens that are their task's successor}; with distil_steps
    also "distil": [...], with beams "answers" (96, beams, answer) and their
    "scores", best first, and "greedy", the greedily decoded tokens."""
    import torch
    gen = torch.Generator(device=device).manual_seed(seed)
    base = layer.KSLinear(PATTERNS, dtype=torch.bfloat16, device=device, seed=seed)
    body = None
    if blocks:
        body = layer.ResidualStack([layer.KSLinear(BLOCK, dtype=torch.bfloat16, device=device, seed=seed + 3 + k)
                                    for k in range(blocks)], base.n_in, post=True, scale=0.5, device=device)
    model = layer.AdapterLinear(base, tasks, rank, alpha=2.0 * rank, seed=seed + 1)
    vocab = base.n_out
    table = torch.randn(vocab, base.n_in, generator=gen, device=device).to(torch.bfloat16)
    successor = torch.stack([torch.randperm(vocab, generator=gen, device=device) for _ in range(tasks)])
    seen = 64                                   # tokens that the answers are made of
    out = {"loss": [], "margin": []}
    if distil_steps:
        for w in base.weights:
            w.requires_grad_(True)
        out["distil"] = distil(base, body, table, distil_steps, lr, state_bits, seed, report)
        for w in base.weights:
            w.requires_grad_(False)

    def vectors(tokens):
        """The model's input for these tokens."""
        if body is None:
            return table[tokens]
        with torch.no_grad():
            return body(table[tokens])

    opt = optim.AdamW(model.parameters(), lr=lr, weight_decay=0.0, state_bits=state_bits, max_norm=1.0, seed=seed)
    for _ in range(steps):
        task = torch.arange(pairs, device=device) % tasks
        task = torch.cat([task, task])[:, None].expand(2 * pairs, tokens)
        inputs = torch.randint(seen, (2 * pairs, tokens), generator=gen, device=device)
        labels = successor[task, inputs]
        labels[pairs:] = torch.randint(vocab, (pairs, tokens), generator=gen, device=device)
        labels[:, 0] = -100                     # the prompt
        ids = task.to(torch.int32).contiguous()
        x = vectors(inputs)
        with torch.no_grad():
            _, ref = libks.sequence_logp(model(x, torch.full_like(ids, -1)), labels)
        opt.zero_grad()
        loss, rewards, _ = layer.preference_loss(model(x, ids), labels, ref, beta=beta)
        loss.backward()
        opt.step()
        out["loss"].append(float(loss.detach()))
        out["margin"].append(float((rewards[:pairs] - rewards[pairs:]).mean()))
        if report:
            report(len(out["loss"]), out["loss"][-1], out["margin"][-1])
    # serving: one token each of requests whose tasks come in any order
    last = torch.randint(seen, (96,), generator=gen, device=device)
    task = torch.randint(tasks, (96,), generator=gen, device=device)
    with torch.no_grad():
        best = model(vectors(last), task.to(torch.int32)).argmax(dim=-1)
    out["correct"] = float((best == successor[task, last]).float().mean())
    if beams:
        def logits_of(tokens):
            ids = task.to(torch.int32)[:, None].expand(tokens.shape)
            return model(vectors(tokens), ids)

        with torch.no_grad():
            out["answers"], out["scores"] = search(logits_of, last, beams, answer)
        out["greedy"] = best
    return out


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--state-bits", type=int, choices=(8, 32), default=8)
    ap.add_argument("--blocks", type=int, default=0, help="KS layers with norms and residuals in front")
    ap.add_argument("--distil-steps", type=int, default=0, help="steps against a dense model's highest logits before")
    ap.add_argument("--beams", type=int, default=0, help="answer by a beam search as well")
    a = ap.parse_args()

    def report(step, loss, margin):
        if step != 1 and step % 10 != 0:
            return
        if margin is None:
            print("distillation step %3d  loss %.4f" % (step, loss), flush=True)
        else:
            print("step %3d  loss %.4f  reward margin %.3f" % (step, loss, margin), flush=True)

    out = run(steps=a.steps, state_bits=a.state_bits, report=report, blocks=a.blocks, distil_steps=a.distil_steps,
              beams=a.beams)
    if a.beams:
        print("first answers:", out["answers"][:3, 0].tolist(), "scores", out["scores"][:3, 0].tolist())
    print("decoded as its task wants: %.0f %% of 96 requests" % (100 * out["correct"]))


if __name__ == "__main__":
    main()
