"""KSLinear: a chain of KS factors as a PyTorch layer, forward and backward
through libks (KS abstract page, taxoreview.com "dblp:303/4794", first
paragraph: the layer built from KS factors; the gradients are the chain rule
on Y = X W^T, see include/ks.h). AdapterLinear: such a layer, frozen, with
low-rank adapters of many requests beside it. preference_loss: the paired
preference loss on token logits.

Argument marshalling only: every product runs in the HIP library. The gradients
are not differentiable themselves: a second derivative raises. With
gradients enabled each factor is its own launch, so that the intermediates
the backward pass needs are kept; without, the chain goes through
``chain_matmul`` and may run fused pairs.
"""
from __future__ import annotations

import functools
import math
from typing import Sequence

from . import libks


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


_LAYER = None
_ADAPTER = None


def __getattr__(name):
    """``layer.KSLinear`` and ``layer.AdapterLinear`` build their class on
    first use (torch is imported lazily, as everywhere in this package)."""
    global _LAYER, _ADAPTER
    if name == "KSLinear":
        if _LAYER is None:
            _LAYER = make_layer_class()
        return _LAYER
    if name == "AdapterLinear":
        if _ADAPTER is None:
            _ADAPTER = make_adapter_class()
        return _ADAPTER
    raise AttributeError(name)
