"""KSLinear: a chain of KS factors as a PyTorch layer, forward and backward
through libks (KS abstract page, taxoreview.com "dblp:303/4794", first
paragraph: the layer built from KS factors; the gradients are the chain rule
on Y = X W^T, see include/ks.h). AdapterLinear: such a layer, frozen, with
low-rank adapters of many requests beside it. ResidualNorm and ResidualStack:
the norms, gates and residuals around such layers. preference_loss and
distillation_loss: the paired preference loss on token logits, and the loss
against a teacher's highest logits.

Argument marshalling only: every product runs in the HIP library. The gradients
are not differentiable themselves: a second derivative raises, and so does a
forward-mode one. With gradients enabled each factor is its own launch, so that
the intermediates the backward pass needs are kept; without, the chain goes
through ``chain_matmul`` and may run fused pairs.
"""
from __future__ import annotations

import functools
import math
from typing import Sequence

from . import libks


def _no_tangents(tensors):
    """Raises if one of a call's tensors(), asked for inside a dual level alone,
    carries a forward-mode tangent, which the library's calls would drop: the
    derivative would read as zero. (An autograd function raises by itself, but a call
    that needs no gradient goes past it.)"""
    import torch
    forward_ad = torch.autograd.forward_ad
    if getattr(forward_ad, "_current_level", 0) < 0:
        return
    if any(t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors()):
        raise NotImplementedError("forward-mode derivatives through libks are not formed")


def _first_only(backward):
    """A backward() whose gradients are constants to autograd: a derivative of one
    raises, where it would silently be zero. (torch's once_differentiable raises
    only if what backward() was given has a derivative, which a loss's 1 has
    not.)"""
    import torch

    class Refuse(torch.autograd.Function):
        @staticmethod
        def forward(ctx, g):
            return g.detach()

        @staticmethod
        def backward(ctx, _):
            raise RuntimeError("a gradient through libks was differentiated: only first derivatives are formed")

    @functools.wraps(backward)
    def call(ctx, *grads):
        _no_tangents(lambda: grads)
        with torch.no_grad():
            out = backward(ctx, *grads)
        if not torch.is_grad_enabled():                # without create_graph
            return out
        return tuple(g if g is None else Refuse.apply(g.requires_grad_()) for g in out)

    return call


def _autograd():
    import torch

    class KSMatmulFunction(torch.autograd.Function):
        """Y = X W^T for one factor; dX = dY W and dK through libks."""

        @staticmethod
        def forward(ctx, X, W, pattern):
            ctx.pattern = tuple(int(v) for v in pattern)
            ctx.save_for_backward(X, W)
            return libks.matmul(X, W, ctx.pattern)

        @staticmethod
        @_first_only
        def backward(ctx, dY):
            X, W = ctx.saved_tensors
            dY = dY.contiguous()
            if dY.dtype != torch.float32:
                dY = dY.float()
            dX = dW = None
            if ctx.needs_input_grad[0]:
                dX = libks.matmul_dx(dY, W, ctx.pattern).to(X.dtype)
            if ctx.needs_input_grad[1]:
                dW = libks.matmul_dw(dY, X, ctx.pattern).to(W.dtype)
            return dX, dW, None

    return KSMatmulFunction


_FN = None


def ks_matmul_autograd(X, W, pattern):
    """Differentiable Y = X W^T for one KS factor (X: (batch, a*c*d))."""
    global _FN
    if _FN is None:
        _FN = _autograd()
    return _FN.apply(X, W, pattern)


def make_layer_class():
    import torch

    class KSLinear(torch.nn.Module):
        """y = x (W_{L-1} ... W_0)^T for KS factors p[0], ..., p[L-1] (applied
        in that order); weights K_k of shape (a, d, b, c), initialised
        N(0, 1/c). Input (..., n_in); output (..., n_out), fp32."""

        def __init__(self, patterns: Sequence[Sequence[int]], dtype=None, device=None, seed: int = 0):
            super().__init__()
            self.patterns = [tuple(int(v) for v in p) for p in patterns]
            for k in range(1, len(self.patterns)):
                a0, b0, _, d0 = self.patterns[k - 1]
                a1, _, c1, d1 = self.patterns[k]
                if a0 * b0 * d0 != a1 * c1 * d1:
                    raise ValueError("factor %d output width does not match factor %d input" % (k - 1, k))
            gen = torch.Generator(device="cpu").manual_seed(seed)
            ws = []
            for (a, b, c, d) in self.patterns:
                w = torch.randn((a, d, b, c), generator=gen) / math.sqrt(c)
                ws.append(torch.nn.Parameter(w.to(device=device, dtype=dtype or torch.float32)))
            self.weights = torch.nn.ParameterList(ws)

        @property
        def n_in(self):
            a, _, c, d = self.patterns[0]
            return a * c * d

        @property
        def n_out(self):
            a, b, _, d = self.patterns[-1]
            return a * b * d

        def forward(self, x):
            lead = x.shape[:-1]
            _no_tangents(lambda: (x, *self.weights))
            x2 = x.reshape(-1, self.n_in).contiguous()
            grad = torch.is_grad_enabled() and (x.requires_grad or any(w.requires_grad for w in self.weights))
            same = all(w.dtype == x2.dtype for w in self.weights) and x2.dtype in (torch.float32, torch.bfloat16)
            if not grad and same:
                y = libks.chain_matmul(x2, list(self.weights), self.patterns)
            else:
                y = x2
                for p, w in zip(self.patterns, self.weights):
                    if not (y.dtype == w.dtype or y.dtype == torch.float32):
                        y = y.float()
                    y = ks_matmul_autograd(y, w, p) if grad else libks.matmul(y, w, p)
            return y.reshape(*lead, self.n_out)

    return KSLinear


def make_adapter_class():
    import torch

    class AdapterFunction(torch.autograd.Function):
        """Y = X W^T + H B^T over an AdapterChain; gradients of X, A and B."""

        @staticmethod
        def forward(ctx, X, A, B, chain, ids):
            Y, H = chain.matmul(X, ids, keep=True)
            ctx.chain = chain
            # the weights are saved for autograd's check of in-place changes: H and the
            # gradients are of the same ones (inference tensors cannot be saved)
            ctx.save_for_backward(X, H, ids, A, B, *(t for t in chain.frozen if not t.is_inference()))
            return Y

        @staticmethod
        @_first_only
        def backward(ctx, dY):
            X, H, ids = ctx.saved_tensors[:3]
            weights = ctx.needs_input_grad[1] or ctx.needs_input_grad[2]
            dX, dA, dB = ctx.chain.backward(dY.float().contiguous(), X, H, ids, weights=weights)
            kind = ctx.chain.weight_dtype
            return (dX.to(X.dtype) if ctx.needs_input_grad[0] else None,
                    dA.to(kind) if ctx.needs_input_grad[1] else None,
                    dB.to(kind) if ctx.needs_input_grad[2] else None, None, None)

    class AdapterLinear(torch.nn.Module):
        """A frozen KSLinear with `adapters` low-rank adapters beside it:
        y = layer(x) + alpha / rank x A[g]^T B[g]^T, where ids gives the
        adapter g of each row (any id outside [0, adapters): none, the layer
        alone). A is drawn N(0, 1/n_in) and B starts at zero, so a new adapter
        changes nothing (more than 1024 rows: nothing beyond rounding). Input
        (..., n_in) with ids (...), int32; output (..., n_out), fp32."""

        def __init__(self, layer, adapters: int, rank: int, alpha: float = 16.0, seed: int = 0):
            super().__init__()
            self.layer = layer
            for w in layer.weights:
                w.requires_grad_(False)
            w = layer.weights[0]
            gen = torch.Generator(device="cpu").manual_seed(seed)
            A = torch.randn((adapters, rank, layer.n_in), generator=gen) / math.sqrt(layer.n_in)
            self.A = torch.nn.Parameter(A.to(device=w.device, dtype=w.dtype))
            self.B = torch.nn.Parameter(torch.zeros((adapters, layer.n_out, rank), device=w.device, dtype=w.dtype))
            self.register_buffer("scale", torch.full((adapters,), alpha / rank, dtype=torch.float32, device=w.device))

        def forward(self, x, ids):
            lead = x.shape[:-1]
            _no_tangents(lambda: (x, self.A, self.B, self.scale, *self.layer.weights))
            x2 = x.reshape(-1, self.layer.n_in).contiguous()
            ids2 = ids.reshape(-1).contiguous()
            # the handle holds addresses, so it is made for the tensors of this call
            chain = libks.AdapterChain([w.detach() for w in self.layer.weights], self.layer.patterns,
                                       self.A.detach(), self.B.detach(), self.scale, transposed=False)
            if torch.is_grad_enabled() and (x2.requires_grad or self.A.requires_grad or self.B.requires_grad):
                y = AdapterFunction.apply(x2, self.A, self.B, chain, ids2)
            else:
                y = chain.matmul(x2, ids2)
            return y.reshape(*lead, self.layer.n_out)

    return AdapterLinear


def make_preference_function():
    import torch

    class PreferenceFunction(torch.autograd.Function):
        """The paired preference loss; its gradient goes to the logits."""

        @staticmethod
        def forward(ctx, logits, labels, ref, beta, smoothing):
            loss, rewards, tokens, scratch = libks._preference_forward(logits, labels, ref, beta, smoothing)
            ctx.save_for_backward(logits, labels, scratch)
            ctx.mark_non_differentiable(rewards, tokens)
            return loss, rewards, tokens

        @staticmethod
        @_first_only
        def backward(ctx, upstream, _rewards, _tokens):
            logits, labels, scratch = ctx.saved_tensors
            return libks._preference_backward(logits, labels, scratch, upstream.float().contiguous()), None, None, \
                None, None

    return PreferenceFunction


_PREFERENCE = None


def preference_loss(logits, labels, ref, beta=0.1, smoothing=0.0):
    """(loss, rewards, tokens) as libks.preference_loss gives them, with the
    loss differentiable in the logits. The gradient is computed in backward(),
    from the logits: they must not be changed in place before it."""
    global _PREFERENCE
    if _PREFERENCE is None:
        _PREFERENCE = make_preference_function()
    return _PREFERENCE.apply(logits, labels, ref, beta, smoothing)


def make_distillation_function():
    import torch

    class DistillationFunction(torch.autograd.Function):
        """The distillation loss; its gradient goes to the student's logits."""

        @staticmethod
        def forward(ctx, logits, labels, ids, top, weight, temperature):
            loss, tokens, stats, _ = libks._on_device(logits.get_device(), libks._distil_forward, logits, labels, ids,
                                                      top, weight, temperature)
            ctx.save_for_backward(logits, labels, ids, top, stats)
            ctx.options = weight, temperature
            ctx.mark_non_differentiable(tokens)
            return loss, tokens

        @staticmethod
        @_first_only
        def backward(ctx, upstream, _tokens):
            logits, labels, ids, top, stats = ctx.saved_tensors
            return libks._on_device(logits.get_device(), libks._distil_backward, logits, labels, ids, top, *ctx.options,
                                    stats, upstream.float().contiguous()), None, None, None, None, None

    return DistillationFunction


_DISTILLATION = None


def distillation_loss(logits, labels, ids, top, weight=1.0, temperature=1.0):
    """(loss, tokens) as libks.distillation_loss gives them, with the loss
    differentiable in the logits (the teacher is a constant). The gradient is
    computed in backward(), from the logits: they must not be changed in place
    before it. libks.distillation_loss forms both at once, in one pass over the
    logits."""
    global _DISTILLATION
    if _DISTILLATION is None:
        _DISTILLATION = make_distillation_function()
    return _DISTILLATION.apply(logits, labels, ids, top, weight, temperature)


def make_norm_classes():
    import torch

    class NormFunction(torch.autograd.Function):
        """(z, h) of a libks.ResidualNorm, h alone without a y; gradients of x, y,
        the gate and the vectors."""

        @staticmethod
        def forward(ctx, norm, dtype, x, y, gate, *vectors):
            z, h, stats = norm.forward(x, y, gate, dtype=dtype, keep=True)
            ctx.norm = norm
            ctx.has = y is not None, gate is not None
            # the vectors too, for autograd's check of in-place changes
            ctx.save_for_backward(x, y, gate, stats, *vectors)
            ctx.set_materialize_grads(False)
            return h if y is None else z if h is None else (z, h)

        @staticmethod
        @_first_only
        def backward(ctx, *grads):
            x, y, gate, stats, *vectors = ctx.saved_tensors
            if y is None:
                dz, dh = None, grads[0]
            else:
                dz, dh = grads if len(grads) == 2 else (grads[0], None)
            dz, dh = (None if g is None else g.contiguous() for g in (dz, dh))
            wanted = ctx.needs_input_grad
            g = ctx.norm.backward(dz, dh, x, y, stats, gate, weights=any(wanted[5:]))
            mine = [None if v is None or d is None else d.to(v.dtype) for v, d in zip(vectors, g[3:])]
            return (None, None, g.dx, g.dy, g.gate, *mine)

    class ResidualNorm(torch.nn.Module):
        """What stands between two blocks: (z, h) = (x + residual scale . gate .
        post(y), pre(z)), with z the residual and h the next block's input. pre and
        post are norms of `kind` "rms" or "layer" (the latter with biases) over the
        last dimension, `scale` a vector that starts at that value; each is left out
        if it is false or None. forward(x, y=None, gate=None): x and y of one shape
        (..., width); without a y, z is x. The gate has x's shape, or that of its first
        dimensions (1 for the others, or none) and width: one for all rows that share
        them. h is of `dtype`, x's by default."""

        def __init__(self, width, kind="rms", pre=True, post=False, scale=None, residual=1.0, eps=1e-6, dtype=None,
                     params=None, device=None):
            super().__init__()
            self.width, self.kind, self.residual, self.eps, self.dtype = int(width), kind, residual, eps, dtype

            def vector(value):
                return torch.nn.Parameter(torch.full((self.width,), float(value), device=device,
                                                     dtype=params or torch.float32))

            bias = kind == "layer"
            self.pre_weight = vector(1) if pre else None
            self.pre_bias = vector(0) if pre and bias else None
            self.post_weight = vector(1) if post else None
            self.post_bias = vector(0) if post and bias else None
            self.scale = vector(scale) if scale is not None else None

        def forward(self, x, y=None, gate=None):
            # of these shapes only are the rows below what they are meant to be: as many
            # values of another shape would be cut into rows as well
            lead = x.shape[:-1]
            if x.shape[-1:] != (self.width,):
                raise ValueError("x must be (..., %d), not %s" % (self.width, tuple(x.shape)))
            if y is not None and y.shape != x.shape:
                raise ValueError("y must have x's shape %s, not %s" % (tuple(x.shape), tuple(y.shape)))

            def rows(t):
                return None if t is None else t.reshape(-1, self.width).contiguous()

            if gate is not None:
                if y is None:
                    raise ValueError("a gate needs a y")
                if gate.shape[-1:] != (self.width,) or gate.dim() > x.dim():
                    raise ValueError("the gate must be (..., %d) with at most x's dimensions, not %s"
                                     % (self.width, tuple(gate.shape)))
                own = list(gate.shape[:-1])
                while own and own[-1] == 1:
                    own.pop()
                if own != list(lead[:len(own)]):
                    raise ValueError("the gate's leading dimensions must be the first of x's")
            vectors = (self.pre_weight, self.pre_bias, self.post_weight, self.post_bias, self.scale)
            x2, y2, gate2 = rows(x), rows(y), rows(gate)
            if y is None and self.pre_weight is None:
                return x, None
            _no_tangents(lambda: (x, y, gate, *vectors))
            # the handle holds addresses, so it is made for the tensors of this call
            norm = libks.ResidualNorm(self.width, *[None if v is None else v.detach() for v in vectors], kind=self.kind,
                                      eps=self.eps, residual=self.residual)
            grad = torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, y, gate, *vectors))
            if not grad:
                z, h = norm.forward(x2, y2, gate2, dtype=self.dtype)
            else:
                out = NormFunction.apply(norm, self.dtype, x2, y2, gate2, *vectors)
                z, h = (x2, out) if y is None else (out, None) if self.pre_weight is None else out
            z = x if y is None else z.reshape(*lead, self.width)
            return z, None if h is None else h.reshape(*lead, self.width)

    class ResidualStack(torch.nn.Module):
        """Blocks (KSLinear, or any modules width -> width) with a residual around
        each: h = pre(x), then z = x + residual scale . gate . post(block(h)) for
        each block in turn, each followed by the norm before the next one in the
        same launch, the last by one more norm. Options as ResidualNorm's. forward(x,
        gates=None): x (..., width), gates one for each block; returns the last
        norm's output."""

        def __init__(self, blocks, width, kind="rms", post=False, scale=None, residual=1.0, eps=1e-6, dtype=None,
                     params=None, device=None):
            super().__init__()
            self.blocks = torch.nn.ModuleList(blocks)
            options = dict(kind=kind, eps=eps, dtype=dtype, params=params, device=device)
            self.first = ResidualNorm(width, **options)
            self.norms = torch.nn.ModuleList(ResidualNorm(width, post=post, scale=scale, residual=residual, **options)
                                             for _ in self.blocks)

        def forward(self, x, gates=None):
            if gates is not None and len(gates) != len(self.blocks):
                raise ValueError("one gate for each block")
            z, h = self.first(x)
            for k, (block, norm) in enumerate(zip(self.blocks, self.norms)):
                z, h = norm(z, block(h), None if gates is None else gates[k])
            return h

    return ResidualNorm, ResidualStack


_LAYER = None
_ADAPTER = None
_NORMS = None


def __getattr__(name):
    """``layer.KSLinear``, ``layer.AdapterLinear``, ``layer.ResidualNorm`` and
    ``layer.ResidualStack`` build their class on first use (torch is imported
    lazily, as everywhere in this package)."""
    global _LAYER, _ADAPTER, _NORMS
    if name == "KSLinear":
        if _LAYER is None:
            _LAYER = make_layer_class()
        return _LAYER
    if name == "AdapterLinear":
        if _ADAPTER is None:
            _ADAPTER = make_adapter_class()
        return _ADAPTER
    if name in ("ResidualNorm", "ResidualStack"):
        if _NORMS is None:
            _NORMS = make_norm_classes()
        return _NORMS[name == "ResidualStack"]
    raise AttributeError(name)
