"""AdamW as a PyTorch optimizer over libks: one launch for every sixty tensors,
moments in fp32 or in 8 bits (include/ks.h, ks_adamw_step). Argument
marshalling only: every value is computed in the HIP library.
"""
from __future__ import annotations

from . import libks


def make_class():
    import torch

    class AdamW(torch.optim.Optimizer):
        """AdamW with decoupled weight decay.

        state_bits: 32 or 8. max_norm: scale the gradients of a step so that
        their norm over all parameters is at most this (a step whose norm is
        not finite changes nothing but its count). seed: of the random rounding
        of 8-bit moments. Parameters and gradients are fp32 or bf16; a
        parameter without a gradient is left alone. 8-bit moments are kept as
        codes and scales, which state_dict() holds as they are."""

        def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, state_bits=32,
                     max_norm=None, seed=0):
            if state_bits not in (8, 32):
                raise ValueError("state_bits must be 8 or 32")
            if max_norm is not None and not max_norm > 0:
                raise ValueError("max_norm must be positive")
            super().__init__(params, dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay))
            self.state_bits, self.max_norm, self.seed = state_bits, max_norm, seed

        def _state(self, p):
            s = self.state[p]
            if not s:
                s["step"] = 0
                if self.state_bits == 32:
                    s["m"] = torch.zeros(p.shape, dtype=torch.float32, device=p.device)
                    s["v"] = torch.zeros_like(s["m"])
                else:
                    s["m"] = torch.zeros(p.shape, dtype=torch.int8, device=p.device)
                    s["v"] = torch.zeros(p.shape, dtype=torch.uint8, device=p.device)
                    s["scales"] = torch.zeros((-(-p.numel() // libks.ADAMW_BLOCK), 2), dtype=torch.float32,
                                              device=p.device)
            return s

        def load_state_dict(self, state_dict):
            # the base class casts floating state to the parameter's type; the
            # moments keep their own
            super().load_state_dict(state_dict)
            saved = state_dict["state"]
            order = [p for g in self.param_groups for p in g["params"]]
            for i, p in enumerate(order):
                for k, x in saved.get(i, {}).items():
                    if isinstance(x, torch.Tensor):
                        self.state[p][k] = x.detach().to(p.device, copy=True)

        @torch.no_grad()
        def step(self, closure=None):
            loss = None
            if closure is not None:
                with torch.enable_grad():
                    loss = closure()
            sets = []       # (options, step, params) with one step number each
            for group in self.param_groups:
                by_step = {}
                for p in group["params"]:
                    if p.grad is not None:
                        by_step.setdefault(self._state(p)["step"] + 1, []).append(p)
                sets += [(group, t, ps) for t, ps in sorted(by_step.items())]
            if not sets:
                return loss

            def handle(ps):
                st = [self.state[p] for p in ps]
                return libks.AdamW([p.detach() for p in ps], [p.grad.contiguous() for p in ps], [s["m"] for s in st],
                                   [s["v"] for s in st], [s["scales"] for s in st] if self.state_bits == 8 else None)

            handles = [handle(ps) for _, _, ps in sets]
            # counted once every tensor has been accepted
            for _, t, ps in sets:
                for p in ps:
                    self.state[p]["step"] = t
            norm = None
            if self.max_norm is not None:
                every = handles[0] if len(handles) == 1 else handle([p for _, _, ps in sets for p in ps])
                norm = every.grad_norm()
            for k, ((group, t, _), h) in enumerate(zip(sets, handles)):
                # another stream of random numbers for each step and set
                seed = (self.seed * 0x9E3779B1 + t * 0xAADDE6A9 + k * 0xBEDE544D) & 0xFFFFFFFF
                h.step(t, group["lr"], group["betas"], group["eps"], group["weight_decay"], self.max_norm, norm, seed)
            return loss

    return AdamW


_CLASS = None


def __getattr__(name):
    """``optim.AdamW`` builds the class on first use (torch is imported
    lazily, as everywhere in this package)."""
    global _CLASS
    if name == "AdamW":
        if _CLASS is None:
            _CLASS = make_class()
        return _CLASS
    raise AttributeError(name)
