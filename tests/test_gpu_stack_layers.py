"""The modules over the residual norm, the distillation loss and beam search
(needs an MI355X): their gradients through autograd against differences and the
64-bit formulas, and the operators together in the training command."""
from __future__ import annotations

import pytest
import torch

import test_gpu_distillation as dist
import test_gpu_residual_norm as norms
from gpu_helpers import DEV, require_gpu
from kronecker_sparse_structured_amd import finetune, layer, libks, optim

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def test_distillation_autograd():
    require_gpu()
    for dtype, V in ((F32, 60), (BF16, 50257), (F32, 70001)):
        x, labels, ids, top = dist.draw(2, 3, V, 9, dtype, seed=11)
        x.requires_grad_(True)
        loss, tokens = layer.distillation_loss(x, labels, ids, top, 0.6, 2.0)
        (2.5 * loss).backward()
        want = dist.formula(x.detach(), labels, ids, top, 0.6, 2.0)
        dist.check((loss.detach(), tokens, x.grad), want, upstream=2.5)
        # at once or in two calls: the same up to the sums' order
        direct = libks.distillation_loss(x.detach(), labels, ids, top, 0.6, 2.0)
        dist.check(direct, want)


def test_distillation_differences():
    require_gpu()
    x, labels, ids, top = dist.draw(2, 4, 50, 6, F32, seed=12)
    x.requires_grad_(True)
    loss, _ = layer.distillation_loss(x, labels, ids, top, 0.6, 2.0)
    loss.backward()
    D = torch.randn(x.shape, generator=torch.Generator().manual_seed(2)).double()
    step = 1e-4
    up, down = (dist.formula(x.detach().double().cpu() + s * step * D, labels, ids, top, 0.6, 2.0)[0][0] for s in (1, -1))
    ana = float((x.grad.double().cpu() * D).sum())
    assert abs((up - down) / (2 * step) - ana) <= 1e-5 * float((x.grad.double().cpu() * D).abs().sum()) + 1e-6


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("gate", [None, "row", "image", "image1", "all"])
def test_residual_norm_module(kind, gate):
    require_gpu()
    B, T, D = 3, 5, 72
    g = torch.Generator().manual_seed(3)
    m = layer.ResidualNorm(D, kind=kind, post=True, scale=0.5, residual=0.8, device=DEV)
    with torch.no_grad():
        for p in m.parameters():
            p.add_(0.2 * torch.randn(D, generator=g).to(DEV))
    x, y = (torch.randn(B, T, D, generator=g).to(DEV).requires_grad_(True) for _ in range(2))
    shape = {None: None, "row": (B, T, D), "image": (B, D), "image1": (B, 1, D), "all": (1, D)}[gate]
    gt = None if shape is None else (1 + torch.randn(shape, generator=g)).to(DEV).requires_grad_(True)
    z, h = m(x, y, gt)
    dz, dh = torch.randn(z.shape, generator=g).to(DEV), torch.randn(h.shape, generator=g).to(DEV)
    ((z * dz).sum() + (h * dh).sum()).backward()
    p = {"x": x.detach().view(-1, D), "y": y.detach().view(-1, D), "kind": kind, "eps": 1e-6, "residual": 0.8,
         "dz": dz.view(-1, D), "dh": dh.view(-1, D), "groups": 0 if gt is None else gt.numel() // D,
         "gate": None if gt is None else gt.detach().view(-1, D), "vectors": {k: None if getattr(m, k) is None else
                                                                             getattr(m, k).detach() for k in norms.VECTORS}}
    got = {"z": z.detach().view(-1, D), "h": h.detach().view(-1, D), "dx": x.grad.view(-1, D), "dy": y.grad.view(-1, D),
           "gate": None if gt is None else gt.grad.view(-1, D)}
    got.update({k: None if getattr(m, k) is None else getattr(m, k).grad for k in norms.VECTORS})
    norms.check(p, got)
    with torch.no_grad():
        z2, h2 = m(x, y, gt)
    assert torch.equal(z2, z) and torch.equal(h2, h)


def test_one_output_and_no_block():
    require_gpu()
    m = layer.ResidualNorm(40, kind="layer", device=DEV)
    x = torch.randn(6, 40, device=DEV, requires_grad=True)
    z, h = m(x)
    assert z is x
    h.sum().backward()
    assert torch.isfinite(x.grad).all() and float(x.grad.abs().max()) < 1e-4     # the mean is taken off
    y = torch.randn(6, 40, device=DEV, requires_grad=True)
    z, _ = m(x, y)
    z.sum().backward()                                                            # h is not used
    assert torch.equal(y.grad, torch.ones_like(y))
    plain = layer.ResidualNorm(40, pre=False, device=DEV)
    assert plain(x)[0] is x and plain(x)[1] is None
    z, h = plain(x, y)
    assert h is None and torch.equal(z, x + y)


def test_gate_shapes_are_checked():
    require_gpu()
    m = layer.ResidualNorm(8, device=DEV)
    x = torch.randn(2, 3, 8, device=DEV)
    for shape in ((3, 8), (1, 3, 8), (2, 2, 8), (2, 3, 4, 8)):
        with pytest.raises(ValueError):
            m(x, x.clone(), torch.ones(shape, device=DEV))
    with pytest.raises(ValueError):
        layer.ResidualStack([torch.nn.Identity()], 8, device=DEV)(x, gates=[])


def test_changed_vectors_are_seen_by_autograd():
    require_gpu()
    m = layer.ResidualNorm(16, device=DEV)
    x, y = (torch.randn(4, 16, device=DEV, requires_grad=True) for _ in range(2))
    z, h = m(x, y)
    with torch.no_grad():
        m.pre_weight.mul_(2)
    with pytest.raises(RuntimeError):
        h.sum().backward()


def test_second_derivatives_raise():
    require_gpu()
    m = layer.ResidualNorm(16, device=DEV)
    x = torch.randn(4, 16, device=DEV, requires_grad=True)
    g, = torch.autograd.grad(m(x)[1].square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
    logits, labels, ids, top = dist.draw(1, 2, 20, 4, F32, seed=1)
    logits.requires_grad_(True)
    g, = torch.autograd.grad(layer.distillation_loss(logits, labels, ids, top)[0], logits, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_stack_against_composed_modules():
    """A stack of KS layers against the same factors, norms and residuals in torch's
    operations in 64 bits."""
    require_gpu()
    blocks = [layer.KSLinear([(4, 8, 8, 2), (1, 8, 8, 8)], device=DEV, seed=k) for k in range(2)]
    stack = layer.ResidualStack(blocks, 64, kind="layer", post=True, scale=0.3, device=DEV)
    x = torch.randn(5, 7, 64, device=DEV, generator=torch.Generator(device=DEV).manual_seed(4), requires_grad=True)
    gates = [torch.rand(5, 64, device=DEV, requires_grad=True) for _ in blocks]
    out = stack(x, gates)
    d = torch.randn(out.shape, device=DEV)
    (out * d).sum().backward()

    def dense(w, p):
        a, b, c, e = p
        m = torch.zeros(a * b * e, a * c * e, dtype=torch.float64, device=DEV)
        i = torch.arange(a * e * b * c, device=DEV)
        ga, be, de, al = i % c, i // c % b, i // (c * b) % e, i // (c * b * e)
        return m.index_put(((al * b + be) * e + de, (al * c + ga) * e + de), w.reshape(-1))

    leaf = {k: v.detach().double().requires_grad_(True) for k, v in
            [*stack.named_parameters(), ("x", x), ("g0", gates[0]), ("g1", gates[1])]}

    def norm(v, name):
        return torch.nn.functional.layer_norm(v, (64,), leaf[name + "_weight"], leaf[name + "_bias"], 1e-6)

    z = leaf["x"]
    h = norm(z, "first.pre")
    for k, block in enumerate(blocks):
        y = h
        for n, p in enumerate(block.patterns):
            y = y @ dense(leaf["blocks.%d.weights.%d" % (k, n)], p).t()
        u = norm(y, "norms.%d.post" % k)
        z = z + leaf["norms.%d.scale" % k] * leaf["g%d" % k][:, None, :] * u
        h = norm(z, "norms.%d.pre" % k)
    (h * d.double()).sum().backward()
    # six norms and four products of 8 terms in fp32, each off by a few 2^-24 of its row's size
    assert float((out.double() - h).norm() / h.norm()) < 1e-5
    for k, v in [*stack.named_parameters(), ("x", x), ("g0", gates[0]), ("g1", gates[1])]:
        assert float((v.grad.double() - leaf[k].grad).norm() / leaf[k].grad.norm()) < 1e-5, k


def test_training_step_of_all_together():
    """Stack, layer, loss and optimizer: a step moves the parameters along the
    gradient that the 64-bit loss of the same logits gives."""
    require_gpu()
    base = layer.KSLinear([(1, 8, 8, 8), (8, 16, 8, 1)], device=DEV, seed=1)
    stack = layer.ResidualStack([layer.KSLinear([(2, 8, 8, 4), (1, 8, 8, 8)], device=DEV, seed=2)], 64, post=True,
                                scale=0.5, device=DEV)
    x = torch.randn(3, 6, 64, device=DEV, generator=torch.Generator(device=DEV).manual_seed(5))
    _, labels, ids, top = dist.draw(3, 6, base.n_out, 8, F32, seed=3)
    params = [*base.parameters(), *stack.parameters()]
    opt = optim.AdamW(params, lr=1e-3, max_norm=1.0)
    losses = []
    for _ in range(3):
        opt.zero_grad()
        logits = base(stack(x))
        loss, tokens = layer.distillation_loss(logits, labels, ids, top, 0.8, 2.0)
        want = dist.formula(logits.detach(), labels, ids, top, 0.8, 2.0)
        dist.check((loss.detach(), tokens, None), want)
        before = [p.detach().clone() for p in params]
        loss.backward()
        assert all(p.grad is not None and torch.isfinite(p.grad).all() for p in params)
        opt.step()
        losses.append(float(loss.detach()))
        assert all(not torch.equal(p, q) for p, q in zip(params, before))
    assert all(l == l for l in losses)


def test_search_with_one_beam_is_greedy_and_more_are_no_worse():
    require_gpu()
    table = torch.randn(300, 300, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    first = torch.arange(20, device=DEV)

    def logits_of(tokens):
        return table[tokens]

    one, score = finetune.search(logits_of, first, 1, 4)
    at = first
    for k in range(4):
        at = table[at].argmax(dim=1)
        assert torch.equal(one[:, 0, k], at)
    log = torch.log_softmax(table.double(), dim=1)
    for beams in (1, 5):
        tokens, scores = finetune.search(logits_of, first, beams, 4)
        at, total = first[:, None].expand(20, beams), torch.zeros(20, beams, dtype=torch.float64, device=DEV)
        for k in range(4):
            total += log[at, tokens[:, :, k]]
            at = tokens[:, :, k]
        # four scores, each off by at most 4e-6 and 42 roundings
        assert float((total - scores).abs().max()) <= 4 * (4e-6 + 42 * 2.0 ** -24 + 2.0 ** -23 * 40)
        assert bool((scores[:, 0] >= score[:, 0] - 1e-4).all())


def test_the_command_with_everything():
    require_gpu()
    out = finetune.run(steps=4, tokens=16, blocks=2, distil_steps=4, beams=3)
    assert len(out["distil"]) == 4 and len(out["loss"]) == 4
    assert all(v == v and abs(v) < 1e6 for v in out["distil"] + out["loss"])
    assert out["answers"].shape == (96, 3, 3) and out["scores"].shape == (96, 3)
    assert bool((out["scores"][:, :-1] >= out["scores"][:, 1:]).all())
    again = finetune.run(steps=4, tokens=16, blocks=2, distil_steps=4, beams=3)
    assert again["distil"] == out["distil"] and again["loss"] == out["loss"]
    assert torch.equal(again["answers"], out["answers"])
    one = finetune.run(steps=2, tokens=16, beams=1, answer=1)
    assert torch.equal(one["answers"][:, 0, 0], one["greedy"])
