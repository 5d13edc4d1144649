"""libks for AMD MI355X: Kronecker-sparse (KS) matrix multiplication.

Y = X W^T where W has support I_a (x) 1_{b x c} (x) I_d and its a*b*c*d
nonzeros are stored as an (a, d, b, c) tensor (KS abstract page,
taxoreview.com "dblp:303/4794", first paragraph). The compute path is the
HIP library libks.so (C ABI in include/ks.h); ``libks`` is its ctypes
binding. Importing this package loads nothing; the first call does.
``layer`` and ``optim`` hold what a model trains with: KS layers, low-rank
adapters beside them, a preference loss and AdamW (``finetune`` runs them
together).
"""
from . import datagen  # noqa: F401  (seeded inputs; no KS arithmetic)

__all__ = ["datagen", "layer", "libks", "optim"]


def __getattr__(name):
    if name in ("layer", "libks", "optim"):
        import importlib
        return importlib.import_module(__name__ + "." + name)
    raise AttributeError(name)
