"""Preference fine-tuning of adapters beside a frozen KS layer, end to end on
synthetic data.

    python -m kronecker_sparse_structured_amd.finetune [--steps 60] [--state-bits 8]

The model is a table of token vectors and one AdapterLinear whose KS factors map
1024 -> 4096; its outputs are the logits of 4096 tokens. There are several
tasks, each with its own adapter: task g wants token t to be followed by a token
of its own. A batch holds pairs of answers of all tasks, the chosen one (the
task's successors) and the rejected one (random tokens); the reference model is
the same layer with the adapters left out (ids -1). Each step runs the adapters
forward and backward, the preference loss with its gradient, and AdamW over the
adapters. At the end one token of each of many requests is decoded in one call,
every row with the adapter of its request.
"""
from __future__ import annotations

import argparse

from . import layer, libks, optim

PATTERNS = [(1, 64, 16, 64), (64, 8, 8, 8)]   # 1024 -> 4096


def run(steps=60, tasks=4, pairs=8, tokens=32, rank=16, state_bits=8, lr=5e-3, beta=0.1, seed=0, device="cuda",
        report=None):
    """Trains and returns {"loss": [...], "margin": [...], "correct": share of
    greedily decoded tokens that are their task's successor}."""
    import torch
    gen = torch.Generator(device=device).manual_seed(seed)
    base = layer.KSLinear(PATTERNS, dtype=torch.bfloat16, device=device, seed=seed)
    model = layer.AdapterLinear(base, tasks, rank, alpha=2.0 * rank, seed=seed + 1)
    vocab = base.n_out
    table = torch.randn(vocab, base.n_in, generator=gen, device=device).to(torch.bfloat16)
    successor = torch.stack([torch.randperm(vocab, generator=gen, device=device) for _ in range(tasks)])
    seen = 64                                   # tokens that the answers are made of
    opt = optim.AdamW(model.parameters(), lr=lr, weight_decay=0.0, state_bits=state_bits, max_norm=1.0, seed=seed)
    out = {"loss": [], "margin": []}
    for _ in range(steps):
        task = torch.arange(pairs, device=device) % tasks
        task = torch.cat([task, task])[:, None].expand(2 * pairs, tokens)
        inputs = torch.randint(seen, (2 * pairs, tokens), generator=gen, device=device)
        labels = successor[task, inputs]
        labels[pairs:] = torch.randint(vocab, (pairs, tokens), generator=gen, device=device)
        labels[:, 0] = -100                     # the prompt
        ids = task.to(torch.int32).contiguous()
        x = table[inputs]
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
        best = model(table[last], task.to(torch.int32)).argmax(dim=-1)
    out["correct"] = float((best == successor[task, last]).float().mean())
    return out


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--state-bits", type=int, choices=(8, 32), default=8)
    a = ap.parse_args()

    def report(step, loss, margin):
        if step == 1 or step % 10 == 0:
            print("step %3d  loss %.4f  reward margin %.3f" % (step, loss, margin), flush=True)

    out = run(steps=a.steps, state_bits=a.state_bits, report=report)
    print("decoded as its task wants: %.0f %% of 96 requests" % (100 * out["correct"]))


if __name__ == "__main__":
    main()
