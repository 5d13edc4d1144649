"""Stack, layer and distillation loss through one backward pass, and the modules'
refusals on tensors of the GPU (needs an MI355X).

The pass is checked in two links. The gradient of the logits against the loss's
formula in 64 bits, with that test's bounds. Then the gradients of all parameters
and of the input against the same factors, norms and residuals in torch's operations
in 64 bits, given the very gradient of the logits that the pass had: what is left is
the rounding of fp32 norms and of products of at most 8 terms, some 2^-24 of a row's
size for each of about 20 of them in a row, 20 to 100 2^-24 = 1e-6 to 6e-6 of a
gradient's norm."""
from __future__ import annotations

import pytest
import torch
from torch.autograd import forward_ad

import test_gpu_distillation as dist
from gpu_helpers import DEV, require_gpu
from kronecker_sparse_structured_amd import layer, optim

pytestmark = pytest.mark.gpu
F32, F64 = torch.float32, torch.float64


def dense(w, p):
    """The matrix of a KS factor, differentiable in its weights."""
    a, b, c, d = p
    m = torch.zeros(a * b * d, a * c * d, dtype=F64, device=w.device)
    i = torch.arange(a * d * b * c, device=w.device)
    ga, be, de, al = i % c, i // c % b, i // (c * b) % d, i // (c * b * d)
    return m.index_put(((al * b + be) * d + de, (al * c + ga) * d + de), w.reshape(-1))


def norm(v, w, b):
    if b is None:
        return v / torch.sqrt(v.square().mean(dim=-1, keepdim=True) + 1e-6) * w
    return torch.nn.functional.layer_norm(v, (v.shape[-1],), w, b, 1e-6)


def chain(h, patterns, leaf, name):
    for n, p in enumerate(patterns):
        h = h @ dense(leaf["%s.weights.%d" % (name, n)], p).t()
    return h


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("w,T", [(0.8, 2.0), (0.6, 1.0), (1.0, 3.0)])
def test_gradients_of_stack_layer_and_loss(kind, w, T):
    require_gpu()
    base = layer.KSLinear([(1, 8, 8, 8), (8, 16, 8, 1)], device=DEV, seed=1)
    blocks = [layer.KSLinear([(2, 8, 8, 4), (1, 8, 8, 8)], device=DEV, seed=2 + k) for k in range(2)]
    stack = layer.ResidualStack(blocks, 64, kind=kind, post=True, scale=0.5, residual=0.7, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn(3, 6, 64, device=DEV, generator=g).requires_grad_(True)
    _, labels, ids, top = dist.draw(3, 6, base.n_out, 8, F32, seed=3)
    params = {**{"base." + k: v for k, v in base.named_parameters()}, **dict(stack.named_parameters())}
    opt = optim.AdamW(list(params.values()), lr=1e-2)
    for _ in range(2):
        opt.zero_grad()
        x.grad = None
        logits = base(stack(x))
        logits.retain_grad()
        loss, tokens = layer.distillation_loss(logits, labels, ids, top, w, T)
        loss.backward()
        dist.check((loss.detach(), tokens, logits.grad), dist.formula(logits.detach(), labels, ids, top, w, T))

        leaf = {k: v.detach().double().requires_grad_(True) for k, v in {**params, "x": x}.items()}
        z = leaf["x"]
        h = norm(z, leaf["first.pre_weight"], leaf.get("first.pre_bias"))
        for k, block in enumerate(blocks):
            u = norm(chain(h, block.patterns, leaf, "blocks.%d" % k), leaf["norms.%d.post_weight" % k],
                     leaf.get("norms.%d.post_bias" % k))
            z = z + 0.7 * leaf["norms.%d.scale" % k] * u
            h = norm(z, leaf["norms.%d.pre_weight" % k], leaf.get("norms.%d.pre_bias" % k))
        out = chain(h, base.patterns, leaf, "base")
        assert float(((logits.detach().double() - out.detach()).norm() / out.detach().norm())) < 1e-5
        out.backward(logits.grad.double())
        for k, v in {**params, "x": x}.items():
            assert float((v.grad.double() - leaf[k].grad).norm() / leaf[k].grad.norm()) < 1e-5, k
        opt.step()                                    # and again from other weights


def test_the_loss_along_its_gradient():
    """Differences of the 64-bit loss of the logits that the layers give, a step up and
    down the gradient of every parameter. A loss is off by its bound el, so a difference
    by 2 el / (2 step) and by the third derivative's step^2; the step is a thousandth of
    the parameters' size, so that its square is 1e-6 of the slope times some tens."""
    require_gpu()
    base = layer.KSLinear([(1, 8, 8, 8), (8, 16, 8, 1)], device=DEV, seed=1)
    stack = layer.ResidualStack([layer.KSLinear([(2, 8, 8, 4), (1, 8, 8, 8)], device=DEV, seed=2)], 64, post=True,
                                scale=0.5, device=DEV)
    x = torch.randn(3, 6, 64, device=DEV, generator=torch.Generator(device=DEV).manual_seed(5))
    _, labels, ids, top = dist.draw(3, 6, base.n_out, 8, F32, seed=3)
    params = [*base.parameters(), *stack.parameters()]
    loss, _ = layer.distillation_loss(base(stack(x)), labels, ids, top, 0.8, 2.0)
    loss.backward()
    size = sum(float(p.detach().double().square().sum()) for p in params) ** 0.5
    slope = sum(float(p.grad.double().square().sum()) for p in params) ** 0.5
    step, values, el = 1e-3 * size / slope, [], 0.0
    start = [p.detach().clone() for p in params]
    for sign in (1, -1):
        moved = 0.0
        with torch.no_grad():
            for p, s in zip(params, start):
                p.copy_(s + sign * step * p.grad)
                moved += float(((p.double() - s.double()) * p.grad.double()).sum())   # the step that fp32 took
            want = dist.formula(base(stack(x)), labels, ids, top, 0.8, 2.0)
        values.append((want[0][0], moved))
        # the logits are off by 1e-5 of their norm, and with them the loss by that times its gradient's share
        el += want[1][0] + 1e-5 * float(want[0][2].norm()) * float(base(stack(x)).detach().double().norm())
    rise, along = values[0][0] - values[1][0], values[0][1] - values[1][1]
    assert along > 0 and abs(rise - along) <= el + 1e-3 * along, (rise, along, el)


def test_refusals_on_the_gpu():
    """The modules' own checks come before the handle's, on the GPU as on the CPU."""
    require_gpu()
    m = layer.ResidualNorm(8, device=DEV)
    x = torch.randn(4, 6, 8, device=DEV)
    for y, gate in ((x, (4, 16)), (x, (24,)), (torch.randn(6, 4, 8, device=DEV), None), (torch.randn(4, 3, 16, device=DEV), None)):
        with pytest.raises(ValueError):
            m(x, y, None if gate is None else torch.ones(gate, device=DEV))
    linear = layer.KSLinear([(1, 4, 2, 4)], device=DEV).requires_grad_(False)
    frozen = layer.ResidualNorm(8, device=DEV).requires_grad_(False)
    logits, labels, ids, top = dist.draw(1, 2, 20, 4, F32, seed=1)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        for call in (frozen, m, linear):
            call(x)
            with pytest.raises(NotImplementedError):
                call(dual)
        with pytest.raises(NotImplementedError):
            layer.distillation_loss(forward_ad.make_dual(logits, torch.ones_like(logits)), labels, ids, top)
    # a gradient whose own derivative is asked for, in the engine's threads
    x.requires_grad_(True)
    z, h = m(x, x)
    with forward_ad.dual_level():
        with pytest.raises(NotImplementedError):
            torch.autograd.grad(h, x, forward_ad.make_dual(torch.ones_like(h), torch.ones_like(h)), retain_graph=True)
