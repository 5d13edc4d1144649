"""Thin Python binding of libks (include/ks.h) through ctypes.

The functions named like the C entry points (``ks_matmul``, ``ks_matmul_ex``,
``ks_chain_workspace_size``, ``ks_chain_matmul``, ``ks_chain_plan``,
``ks_chain_describe``, ``ks_plan_describe``, ``ks_status_string``,
``ks_version``, the gradient calls) only marshal arguments: tensors become
device pointers, the stream defaults to torch's current stream, and a
non-OK status raises ``KSError``. Every step of the computation runs in the
HIP kernels of libks.so; there is no fallback. If the library is not built,
loading fails loudly.

``matmul`` and ``chain_matmul`` are conveniences over the same calls that
allocate the output (and the chain workspace) with torch. They, the adapters,
the preference loss and the optimizer count what they write into a caller's
tensor as an in-place change (torch's version counter), so that autograd sees
it; the ``ks_`` calls write through addresses and do not. Their ``stream``
(default: torch's current one) is the one that the call launches on and
allocates for.
"""
from __future__ import annotations

import array
import ctypes
import operator
import os
from typing import Optional, Sequence

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libks.so")

# ks_dtype_t
DTYPE_F32, DTYPE_BF16, DTYPE_BF16W = 0, 1, 2
# ks_kernel_t
KERNEL_AUTO, KERNEL_GENERIC, KERNEL_VALU, KERNEL_MFMA, KERNEL_MFMA_LDS, KERNEL_COLUMN = 0, 1, 2, 3, 4, 5
KERNELS = {"auto": KERNEL_AUTO, "generic": KERNEL_GENERIC, "valu": KERNEL_VALU, "mfma": KERNEL_MFMA,
           "mfma_lds": KERNEL_MFMA_LDS, "col": KERNEL_COLUMN}
# ks_store_waves_t
STORE_AUTO, STORE_COMPUTE, STORE_DEDICATED = 0, 1, 2
STORE_WAVES = {"auto": STORE_AUTO, "compute": STORE_COMPUTE, "dedicated": STORE_DEDICATED}
# chain flags
CHAIN_AUTO, CHAIN_NO_FUSE = 0, 1
# ks_status_t
STATUS = ["KS_OK", "KS_ERR_NULL", "KS_ERR_PATTERN", "KS_ERR_BATCH", "KS_ERR_DTYPE",
          "KS_ERR_CHAIN_MISMATCH", "KS_ERR_WORKSPACE", "KS_ERR_ALIGN", "KS_ERR_OVERLAP",
          "KS_ERR_HIP", "KS_ERR_UNSUPPORTED", "KS_ERR_INVALID"]
for _i, _n in enumerate(STATUS):
    globals()[_n] = _i


class KSError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s" % (where, ks_status_string(status)))


class ks_pattern_t(ctypes.Structure):
    _fields_ = [("a", ctypes.c_int32), ("b", ctypes.c_int32),
                ("c", ctypes.c_int32), ("d", ctypes.c_int32)]


MFMA_TILES = 7   # KS_MFMA_TILES: tile candidates of the matrix-core kernel


class ks_options_t(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int32), ("rows_per_block", ctypes.c_int32),
                ("store_waves", ctypes.c_int32), ("mfma_tile", ctypes.c_int32), ("mfma_loaders", ctypes.c_int32),
                ("reserved", ctypes.c_int32 * 3)]


class ks_closure_t(ctypes.Structure):
    _fields_ = [("components", ctypes.c_int64), ("mid", ctypes.c_int64), ("inputs", ctypes.c_int64),
                ("outputs", ctypes.c_int64), ("weights", ctypes.c_int64), ("in_run", ctypes.c_int64),
                ("out_run", ctypes.c_int64), ("tile_components", ctypes.c_int64), ("tile_weights", ctypes.c_int64),
                ("uniform", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class ks_adapters_t(ctypes.Structure):
    _fields_ = [("A", ctypes.c_void_p), ("B", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("n_in", ctypes.c_int64), ("n_out", ctypes.c_int64),
                ("rank", ctypes.c_int32), ("count", ctypes.c_int32)]


class ks_logits_t(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("labels", ctypes.c_void_p),
                ("seq_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64), ("label_stride", ctypes.c_int64),
                ("sequences", ctypes.c_int64), ("tokens", ctypes.c_int64), ("vocab", ctypes.c_int64),
                ("elem", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class ks_adamw_tensor_t(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("g", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("p_elem", ctypes.c_int32), ("g_elem", ctypes.c_int32)]


class ks_adamw_options_t(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("max_norm", ctypes.c_double),
                ("step", ctypes.c_int64), ("seed", ctypes.c_uint32), ("state_bits", ctypes.c_int32)]


# ks_elem_t
ELEM_F32, ELEM_BF16 = 0, 1

_lib = None


def _hip_runtimes() -> set:
    """Paths of the HIP runtime libraries mapped into this process."""
    try:
        with open("/proc/self/maps") as f:
            return {line.split()[-1] for line in f
                    if len(line.split()) >= 6 and "libamdhip64.so" in line.split()[-1]}
    except OSError:
        return set()


def load(path: str = LIB_PATH):
    """Load libks.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise FileNotFoundError(
            "libks.so not found at %s; build it with "
            "`python -m kronecker_sparse_structured_amd.build`" % path)
    # torch ships its own copy of the HIP runtime. Load it first so that
    # libks binds to that copy: with two runtimes in one process, pointers
    # and streams from torch are unknown to the one libks calls.
    import torch  # noqa: F401
    lib = ctypes.CDLL(path)
    runtimes = _hip_runtimes()
    if len(runtimes) > 1:
        raise RuntimeError("more than one HIP runtime is loaded in this process (%s); "
                           "libks must share torch's" % ", ".join(sorted(runtimes)))
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.ks_status_string.argtypes = [i32]
    lib.ks_status_string.restype = ctypes.c_char_p
    lib.ks_version.argtypes = []
    lib.ks_version.restype = ctypes.c_char_p
    lib.ks_matmul.argtypes = [ks_pattern_t, vp, vp, vp, i64, i32, vp]
    lib.ks_matmul.restype = i32
    lib.ks_matmul_ex.argtypes = [ks_pattern_t, vp, vp, vp, i64, i32, vp, ctypes.POINTER(ks_options_t)]
    lib.ks_matmul_ex.restype = i32
    lib.ks_chain_workspace_size.argtypes = [ctypes.POINTER(ks_pattern_t), i32, i64, i32,
                                            ctypes.c_uint, ctypes.POINTER(ctypes.c_size_t)]
    lib.ks_chain_workspace_size.restype = i32
    lib.ks_chain_matmul.argtypes = [ctypes.POINTER(ks_pattern_t), i32, ctypes.POINTER(vp), vp, vp,
                                    i64, i32, vp, ctypes.c_size_t, ctypes.c_uint, vp]
    lib.ks_chain_matmul.restype = i32
    lib.ks_chain_plan.argtypes = [ctypes.POINTER(ks_pattern_t), i32, i64, i32, ctypes.c_uint,
                                  ctypes.POINTER(ctypes.c_int), i32, ctypes.POINTER(ctypes.c_int)]
    lib.ks_chain_plan.restype = i32
    lib.ks_plan_describe.argtypes = [ks_pattern_t, i64, i32, ctypes.c_char_p, ctypes.c_size_t]
    lib.ks_plan_describe.restype = i32
    lib.ks_chain_describe.argtypes = [ctypes.POINTER(ks_pattern_t), i32, i64, i32, ctypes.c_uint,
                                      ctypes.c_char_p, ctypes.c_size_t]
    lib.ks_chain_describe.restype = i32
    lib.ks_pair_closure.argtypes = [ks_pattern_t, ks_pattern_t, ctypes.POINTER(ks_closure_t)]
    lib.ks_pair_closure.restype = i32
    lib.ks_matmul_dx_workspace_size.argtypes = [ks_pattern_t, i32, ctypes.POINTER(ctypes.c_size_t)]
    lib.ks_matmul_dx_workspace_size.restype = i32
    lib.ks_matmul_dx.argtypes = [ks_pattern_t, vp, vp, vp, i64, i32, vp, ctypes.c_size_t, vp]
    lib.ks_matmul_dx.restype = i32
    lib.ks_matmul_dw_workspace_size.argtypes = [ks_pattern_t, i64, i32, ctypes.POINTER(ctypes.c_size_t)]
    lib.ks_matmul_dw_workspace_size.restype = i32
    lib.ks_matmul_dw.argtypes = [ks_pattern_t, vp, vp, vp, i64, i32, vp, ctypes.c_size_t, vp]
    lib.ks_matmul_dw.restype = i32
    lib.ks_matmul_dw_noalloc.argtypes = [ks_pattern_t, vp, vp, vp, i64, i32, vp]
    lib.ks_matmul_dw_noalloc.restype = i32
    pp, pa, pl, pt = (ctypes.POINTER(t) for t in (ks_pattern_t, ks_adapters_t, ks_logits_t, ks_adamw_tensor_t))
    f32, size, psize = ctypes.c_float, ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t)
    for name, args in {
        "ks_adapter_workspace_size": [pa, i64, psize],
        "ks_adapter_matmul": [pa, vp, vp, vp, vp, i64, i32, vp, size, vp],
        "ks_adapter_backward_workspace_size": [pa, i64, psize],
        "ks_adapter_backward": [pa, vp, vp, vp, vp, vp, vp, vp, i64, i32, vp, size, vp],
        "ks_chain_adapter_workspace_size": [pp, i32, pa, i64, i32, psize],
        "ks_chain_adapter_matmul": [pp, i32, ctypes.POINTER(vp), pa, vp, vp, vp, vp, i64, i32, vp, size, vp],
        "ks_chain_transpose_size": [pp, i32, i32, psize],
        "ks_chain_transpose": [pp, i32, ctypes.POINTER(vp), vp, i32, vp],
        "ks_chain_adapter_backward_workspace_size": [pp, i32, pa, i64, i32, i32, psize],
        "ks_chain_adapter_backward": [pp, i32, ctypes.POINTER(vp), vp, pa, vp, vp, vp, vp, vp, vp, vp, i64, i32, vp, size,
                                      vp],
        "ks_sequence_logp": [pl, vp, vp, vp, vp],
        "ks_preference_loss": [pl, vp, i64, f32, f32, vp, vp, vp, vp, vp, vp, i64, i64, vp],
        "ks_preference_backward": [pl, vp, vp, vp, vp, i64, i64, vp],
        "ks_grad_norm_workspace_size": [pt, i32, psize],
        "ks_grad_norm": [pt, i32, vp, vp, size, vp],
        "ks_adamw_step": [pt, i32, ctypes.POINTER(ks_adamw_options_t), vp, vp],
        "ks_adamw_state_values": [pt, i32, ctypes.POINTER(vp), ctypes.POINTER(vp), vp],
    }.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = i32
    _lib = lib
    return lib


# ---------------------------------------------------------------- marshalling

def _pattern(p) -> ks_pattern_t:
    if isinstance(p, ks_pattern_t):
        return p
    a, b, c, d = (int(v) for v in p)
    return ks_pattern_t(a, b, c, d)


def _ptr(x) -> Optional[int]:
    """Device address of a tensor, or an int address, or None (NULL)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return int(x.data_ptr())


def _stream(stream, *tensors) -> Optional[int]:
    if stream is None:
        import torch
        for t in tensors:
            if t is not None and not isinstance(t, int) and t.is_cuda:
                return int(torch.cuda.current_stream(t.device).cuda_stream)
        return None
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def _raw_stream(index: int):
    """Torch's current stream of a device index (no stream object where torch has
    the handle at hand)."""
    import torch
    get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return get(index) if get is not None else int(torch.cuda.current_stream(index).cuda_stream)


def _on_stream(stream, device, call, *args):
    """call(*args) with `stream` (a stream object or its address) as torch's
    current one. What the call allocates then comes from that stream's memory:
    a workspace that it drops goes to nobody else before its kernels are done.
    Results are held for the caller's current stream as well, which may read
    them once it has waited for `stream`. Tensors that the caller gives are the
    caller's to keep until then."""
    import torch
    raw = stream if isinstance(stream, int) else int(stream.cuda_stream)
    here = torch.cuda.current_stream(device)
    if raw == here.cuda_stream:
        return call(*args)
    with torch.cuda.stream(torch.cuda.ExternalStream(raw, device=device)):
        out = call(*args)
    for t in out if isinstance(out, tuple) else (out,):
        if t is not None:
            t.record_stream(here)
    return out


def _raise(status: int, where: str, check: bool) -> int:
    if check and status != 0:
        raise KSError(status, where)
    return status


# ---------------------------------------------------------------- C entry points

def ks_status_string(status: int) -> str:
    return load().ks_status_string(int(status)).decode()


def ks_version() -> str:
    return load().ks_version().decode()


def ks_matmul(p, W, X, Y, batch: int, dtype: int, stream=None, check: bool = True) -> int:
    st = load().ks_matmul(_pattern(p), _ptr(W), _ptr(X), _ptr(Y), int(batch), int(dtype),
                          _stream(stream, Y, X, W))
    return _raise(st, "ks_matmul", check)


def ks_matmul_ex(p, W, X, Y, batch: int, dtype: int, stream=None, kernel: int = KERNEL_AUTO,
                 rows_per_block: int = 0, check: bool = True, reserved=None, store_waves=STORE_AUTO,
                 mfma_tile: int = 0, mfma_loaders: int = 0) -> int:
    opt = ks_options_t()
    opt.kernel = KERNELS.get(kernel, kernel) if isinstance(kernel, str) else int(kernel)
    opt.rows_per_block = int(rows_per_block)
    opt.mfma_tile = int(mfma_tile)
    opt.mfma_loaders = int(mfma_loaders)
    opt.store_waves = STORE_WAVES.get(store_waves, store_waves) if isinstance(store_waves, str) else int(store_waves)
    if reserved is not None:
        for i, v in enumerate(reserved):
            opt.reserved[i] = int(v)
    st = load().ks_matmul_ex(_pattern(p), _ptr(W), _ptr(X), _ptr(Y), int(batch), int(dtype),
                             _stream(stream, Y, X, W), ctypes.byref(opt))
    return _raise(st, "ks_matmul_ex", check)


def ks_matmul_dx_workspace_size(p, dtype: int, check: bool = True):
    out = ctypes.c_size_t(0)
    st = load().ks_matmul_dx_workspace_size(_pattern(p), int(dtype), ctypes.byref(out))
    _raise(st, "ks_matmul_dx_workspace_size", check)
    return out.value if check else (st, out.value)


def ks_matmul_dx(p, W, dY, dX, batch: int, dtype: int, ws, ws_bytes: int, stream=None, check: bool = True) -> int:
    st = load().ks_matmul_dx(_pattern(p), _ptr(W), _ptr(dY), _ptr(dX), int(batch), int(dtype), _ptr(ws),
                             int(ws_bytes), _stream(stream, dX, dY, W))
    return _raise(st, "ks_matmul_dx", check)


def ks_matmul_dw_workspace_size(p, batch: int, dtype: int, check: bool = True):
    out = ctypes.c_size_t(0)
    st = load().ks_matmul_dw_workspace_size(_pattern(p), int(batch), int(dtype), ctypes.byref(out))
    _raise(st, "ks_matmul_dw_workspace_size", check)
    return out.value if check else (st, out.value)


def ks_matmul_dw(p, dY, X, dW, batch: int, dtype: int, ws, ws_bytes: int, stream=None, check: bool = True) -> int:
    st = load().ks_matmul_dw(_pattern(p), _ptr(dY), _ptr(X), _ptr(dW), int(batch), int(dtype), _ptr(ws),
                             int(ws_bytes), _stream(stream, dW, dY, X))
    return _raise(st, "ks_matmul_dw", check)


def ks_matmul_dw_noalloc(p, dY, X, dW, batch: int, dtype: int, stream=None, check: bool = True) -> int:
    st = load().ks_matmul_dw_noalloc(_pattern(p), _ptr(dY), _ptr(X), _ptr(dW), int(batch), int(dtype),
                                     _stream(stream, dW, dY, X))
    return _raise(st, "ks_matmul_dw_noalloc", check)


def _patterns(ps: Sequence):
    arr = (ks_pattern_t * max(len(ps), 1))()
    for i, p in enumerate(ps):
        arr[i] = _pattern(p)
    return arr


def ks_chain_workspace_size(ps: Sequence, batch: int, dtype: int, flags: int = CHAIN_AUTO,
                            n: Optional[int] = None, check: bool = True):
    """Returns the workspace size in bytes (or (status, size) if check=False)."""
    out = ctypes.c_size_t(0)
    st = load().ks_chain_workspace_size(_patterns(ps), len(ps) if n is None else n, int(batch),
                                        int(dtype), int(flags), ctypes.byref(out))
    if not check:
        return st, out.value
    _raise(st, "ks_chain_workspace_size", True)
    return out.value


def ks_chain_matmul(ps: Sequence, Ws: Sequence, X, Y, batch: int, dtype: int, ws=None,
                    ws_bytes: int = 0, flags: int = CHAIN_AUTO, stream=None,
                    n: Optional[int] = None, check: bool = True) -> int:
    wp = (ctypes.c_void_p * max(len(Ws), 1))(*[_ptr(w) for w in Ws])
    st = load().ks_chain_matmul(_patterns(ps), len(ps) if n is None else n, wp, _ptr(X), _ptr(Y),
                                int(batch), int(dtype), _ptr(ws), int(ws_bytes), int(flags),
                                _stream(stream, Y, X))
    return _raise(st, "ks_chain_matmul", check)


def ks_chain_plan(ps: Sequence, batch: int, dtype: int, flags: int = CHAIN_AUTO) -> list:
    """Group lengths of a chain's launches (1 = single factor, 2 = fused pair or a
    run of two, more = a row-resident run)."""
    cap = max(len(ps), 1)
    lens = (ctypes.c_int * cap)()
    ng = ctypes.c_int(0)
    _raise(load().ks_chain_plan(_patterns(ps), len(ps), int(batch), int(dtype), int(flags), lens, cap,
                                ctypes.byref(ng)), "ks_chain_plan", True)
    return [lens[i] for i in range(ng.value)]


def ks_chain_groups(ps: Sequence, batch: int, dtype: int, flags: int = CHAIN_AUTO) -> list:
    """Factor indices of each launch group, e.g. [[0, 1], [2], [3]]."""
    out, k = [], 0
    for ln in ks_chain_plan(ps, batch, dtype, flags):
        out.append(list(range(k, k + ln)))
        k += ln
    return out


def ks_pair_closure(f, g) -> dict:
    """The closure rule for running factor f then g in one pass (ks.h)."""
    out = ks_closure_t()
    _raise(load().ks_pair_closure(_pattern(f), _pattern(g), ctypes.byref(out)), "ks_pair_closure", True)
    return {name: int(getattr(out, name)) for name, _ in ks_closure_t._fields_ if name != "reserved"}


def ks_chain_describe(ps: Sequence, batch: int, dtype: int, flags: int = CHAIN_AUTO) -> str:
    """The kernel of each launch group, "[first..last] description; ..."."""
    buf = ctypes.create_string_buffer(4096)
    _raise(load().ks_chain_describe(_patterns(ps), len(ps), int(batch), int(dtype), int(flags), buf, 4096),
           "ks_chain_describe", True)
    return buf.value.decode()


def ks_plan_describe(p, batch: int, dtype: int) -> str:
    buf = ctypes.create_string_buffer(512)
    _raise(load().ks_plan_describe(_pattern(p), int(batch), int(dtype), buf, 512), "ks_plan_describe", True)
    return buf.value.decode()


# ---------------------------------------------------------------- conveniences

def dtype_code(x_dtype, w_dtype) -> int:
    import torch
    if x_dtype == torch.float32 and w_dtype == torch.float32:
        return DTYPE_F32
    if x_dtype == torch.bfloat16 and w_dtype == torch.bfloat16:
        return DTYPE_BF16
    if x_dtype == torch.float32 and w_dtype == torch.bfloat16:
        return DTYPE_BF16W
    raise TypeError("unsupported dtypes X=%s W=%s" % (x_dtype, w_dtype))


def _check_tensor(t, name):
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _wrote(tensors):
    """Counts a write through their addresses as an in-place change of these
    tensors (one, or several), as an operation of torch's own would. Without it
    autograd would take a changed tensor for the one it saved."""
    import torch
    torch.autograd.graph.increment_version(tensors)


def matmul(X, W, pattern, out=None, kernel="auto", stream=None):
    """Y = X W^T for one KS factor; X is (batch, a*c*d), W is (a, d, b, c)."""
    import torch
    a, b, c, d = (int(v) for v in pattern)
    _check_tensor(X, "X")
    _check_tensor(W, "W")
    if X.dim() != 2 or X.shape[1] != a * c * d:
        raise ValueError("X must be (batch, a*c*d) = (*, %d)" % (a * c * d))
    if W.numel() != a * b * c * d:
        raise ValueError("W must hold a*b*c*d = %d values" % (a * b * c * d))
    if stream is not None:
        return _on_stream(stream, X.device, matmul, X, W, pattern, out, kernel)
    batch = X.shape[0]
    given = out is not None
    if not given:
        out = torch.empty((batch, a * b * d), dtype=torch.float32, device=X.device)
    ks_matmul_ex((a, b, c, d), W, X, out, batch, dtype_code(X.dtype, W.dtype), kernel=kernel)
    if given:
        _wrote(out)
    return out


def chain_matmul(X, Ws, patterns, out=None, fuse=True, stream=None):
    """Apply the factors in order (factor 0 first); returns fp32 Y."""
    import torch
    _check_tensor(X, "X")
    for i, w in enumerate(Ws):
        _check_tensor(w, "W[%d]" % i)
    if stream is not None:
        return _on_stream(stream, X.device, chain_matmul, X, Ws, patterns, out, fuse)
    dt = dtype_code(X.dtype, Ws[0].dtype)
    batch = X.shape[0]
    last = patterns[-1]
    given = out is not None
    if not given:
        out = torch.empty((batch, int(last[0]) * int(last[1]) * int(last[3])),
                          dtype=torch.float32, device=X.device)
    flags = CHAIN_AUTO if fuse else CHAIN_NO_FUSE
    nbytes = ks_chain_workspace_size(patterns, batch, dt, flags)
    ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=X.device) if nbytes else None
    ks_chain_matmul(patterns, Ws, X, out, batch, dt, ws, nbytes, flags)
    if given:
        _wrote(out)
    return out


def matmul_dx(dY, W, pattern, out=None, stream=None):
    """dX = dY W for one KS factor (the gradient of matmul with respect to X)."""
    import torch
    a, b, c, d = (int(v) for v in pattern)
    _check_tensor(dY, "dY")
    _check_tensor(W, "W")
    if dY.dim() != 2 or dY.shape[1] != a * b * d:
        raise ValueError("dY must be (batch, a*b*d) = (*, %d)" % (a * b * d))
    if stream is not None:
        return _on_stream(stream, dY.device, matmul_dx, dY, W, pattern, out)
    batch = dY.shape[0]
    dt = dtype_code(dY.dtype, W.dtype)
    given = out is not None
    if not given:
        out = torch.empty((batch, a * c * d), dtype=torch.float32, device=dY.device)
    nbytes = ks_matmul_dx_workspace_size((a, b, c, d), dt)
    ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dY.device)
    ks_matmul_dx((a, b, c, d), W, dY, out, batch, dt, ws, nbytes)
    if given:
        _wrote(out)
    return out


def matmul_dw(dY, X, pattern, out=None, stream=None):
    """dK (shape (a, d, b, c), fp32): the gradient of matmul with respect to W."""
    import torch
    a, b, c, d = (int(v) for v in pattern)
    _check_tensor(dY, "dY")
    _check_tensor(X, "X")
    if dY.dtype != torch.float32:
        raise TypeError("dY must be fp32")
    if X.dim() != 2 or X.shape[1] != a * c * d or dY.shape != (X.shape[0], a * b * d):
        raise ValueError("X must be (batch, a*c*d) and dY (batch, a*b*d)")
    if stream is not None:
        return _on_stream(stream, dY.device, matmul_dw, dY, X, pattern, out)
    batch = X.shape[0]
    dt = DTYPE_BF16 if X.dtype == torch.bfloat16 else DTYPE_F32
    given = out is not None
    if not given:
        out = torch.empty((a, d, b, c), dtype=torch.float32, device=X.device)
    nbytes = ks_matmul_dw_workspace_size((a, b, c, d), batch, dt)
    ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=X.device) if nbytes else None
    ks_matmul_dw((a, b, c, d), dY, X, out, batch, dt, ws, nbytes)
    if given:
        _wrote(out)
    return out


# ---------------------------------------------------------------- adapters

class AdapterChain:
    """A chain of KS factors with low-rank adapters of many requests beside it:
    Y[n] = X[n] W^T + H[n] B[g]^T, H[n] = scale[g] X[n] A[g]^T, g = ids[n]
    (no adapter for an id outside [0, G)).

    The handle keeps its weights and their addresses, so that a call only
    marshals its rows; later in-place changes of them are seen. With `transposed`
    it also keeps W's blocks transposed, for the backward() calls of a training
    loop: made here once, where each call makes its own otherwise, and left unused
    after an in-place operation on a W that torch counts, this module's optimizer
    among them. Changes that torch does not count (through W.data, by a replayed
    graph, by code that writes through W's address) need a new handle; inference
    tensors have no such count, and each call transposes them. W_k has shape (a, d, b, c); A (G, rank, n_in); B (G,
    n_out, rank); scale (G,) fp32; W, A and B have one type, fp32 or bf16; X has
    that type, or is fp32."""

    def __init__(self, Ws, patterns, A, B, scale, transposed=False):
        import torch
        self.patterns = [tuple(int(v) for v in p) for p in patterns]
        if not self.patterns or len(Ws) != len(self.patterns):
            raise ValueError("one weight tensor for each pattern, at least one")
        for i, (w, p) in enumerate(zip(Ws, self.patterns)):
            _check_tensor(w, "W[%d]" % i)
            if w.numel() != p[0] * p[1] * p[2] * p[3]:
                raise ValueError("W[%d] must hold a*b*c*d = %d values" % (i, p[0] * p[1] * p[2] * p[3]))
        for t, name in ((A, "A"), (B, "B"), (scale, "scale")):
            _check_tensor(t, name)
        first, last = self.patterns[0], self.patterns[-1]
        self.n_in, self.n_out = first[0] * first[2] * first[3], last[0] * last[1] * last[3]
        if A.dim() != 3 or A.shape[2] != self.n_in:
            raise ValueError("A must be (adapters, rank, %d)" % self.n_in)
        self.count, self.rank = int(A.shape[0]), int(A.shape[1])
        if tuple(B.shape) != (self.count, self.n_out, self.rank):
            raise ValueError("B must be (%d, %d, %d)" % (self.count, self.n_out, self.rank))
        if tuple(scale.shape) != (self.count,) or scale.dtype != torch.float32:
            raise ValueError("scale must be (%d,) fp32" % self.count)
        if any(t.dtype != A.dtype for t in (*Ws, B)):
            raise TypeError("W, A and B must have one type")
        self.device = A.device
        if any(t.device != self.device for t in (*Ws, B, scale)):
            raise ValueError("all weights must be on one device")
        self.weight_dtype = A.dtype
        self._codes = {torch.float32: dtype_code(torch.float32, A.dtype)}
        if A.dtype == torch.bfloat16:
            self._codes[torch.bfloat16] = DTYPE_BF16
        self._keep = (list(Ws), A, B, scale)
        self.frozen = (*Ws, scale)           # what backward() reads and gives no gradient of
        self._f32 = scale.new_empty          # an fp32 tensor beside the weights, without torch.empty's keywords
        self._n = len(self.patterns)
        self._p = _patterns(self.patterns)
        self._w = (ctypes.c_void_p * self._n)(*[w.data_ptr() for w in Ws])
        self._ad = ks_adapters_t(A.data_ptr(), B.data_ptr(), scale.data_ptr(), self.n_in, self.n_out, self.rank,
                                 self.count)
        self._lib = load()
        self._index = A.get_device()
        self._sizes = {}
        self._wt = self._versions = None
        # inference tensors have no version to tell a change by
        if transposed and not torch.cuda.is_current_stream_capturing() and not any(w.is_inference() for w in Ws):
            code, size = self._codes[torch.float32], ctypes.c_size_t(0)
            _raise(self._lib.ks_chain_transpose_size(self._p, self._n, code, size), "ks_chain_transpose_size", True)
            self._wt = torch.empty(size.value, dtype=torch.uint8, device=self.device)
            self._versions = [w._version for w in Ws]
            _raise(self._lib.ks_chain_transpose(self._p, self._n, self._w, self._wt.data_ptr(), code,
                                                _raw_stream(self._index)), "ks_chain_transpose", True)
            # calls may come on any stream
            torch.cuda.current_stream(self._index).synchronize()
            self._wt_stream = _raw_stream(self._index)

    def _workspace(self, name, batch, *args):
        """A workspace and its size; the size of a batch is asked for once."""
        key = (name, batch, *args)
        n = self._sizes.get(key)
        if n is None:
            size = ctypes.c_size_t(0)
            _raise(getattr(self._lib, name)(self._p, self._n, self._ad, batch, *args, size), name, True)
            if len(self._sizes) > 256:
                self._sizes.clear()
            n = self._sizes[key] = size.value
        if n == 0:
            return None, 0, None
        ws = self._f32((n + 3) // 4)
        return ws.data_ptr(), n, ws

    def _rows(self, X, ids):
        import torch
        if X.dim() != 2 or X.shape[1] != self.n_in:
            raise ValueError("X must be (batch, %d)" % self.n_in)
        if ids.dtype != torch.int32 or tuple(ids.shape) != (X.shape[0],):
            raise ValueError("ids must be (batch,) int32")
        if X.get_device() != self._index or ids.get_device() != self._index:
            raise ValueError("X and ids must be on the weights' device")
        if not X.is_contiguous() or not ids.is_contiguous():
            raise ValueError("X and ids must be contiguous")
        code = self._codes.get(X.dtype)
        if code is None:
            raise TypeError("X must be fp32 or of the weights' type, not %s" % X.dtype)
        return X.shape[0], code

    def matmul(self, X, ids, out=None, keep=False, stream=None):
        """Y (batch, n_out) fp32; with keep=True (Y, H), H (batch, rank) fp32
        for backward()."""
        import torch
        if stream is not None:
            return _on_stream(stream, self.device, self.matmul, X, ids, out, keep)
        batch, code = self._rows(X, ids)
        given = out is not None
        if not given:
            out = self._f32(batch, self.n_out)
        else:
            _check_out(out, (batch, self.n_out), torch.float32, self.device, "out")
        H = self._f32(batch, self.rank) if keep else None
        ws, size, _keep = self._workspace("ks_chain_adapter_workspace_size", batch, code)
        _raise(self._lib.ks_chain_adapter_matmul(
            self._p, self._n, self._w, self._ad, ids.data_ptr(), X.data_ptr(), out.data_ptr(), _ptr(H), batch, code,
            ws, size, _raw_stream(self._index)), "ks_chain_adapter_matmul", True)
        if given:
            _wrote(out)
        return (out, H) if keep else out

    def backward(self, dY, X, H, ids, weights=True, stream=None):
        """(dX, dA, dB), all fp32; (dX, None, None) with weights=False. W is
        frozen. dY (batch, n_out) fp32; X, H and ids as matmul() had and gave
        them."""
        import torch
        if stream is not None:
            return _on_stream(stream, self.device, self.backward, dY, X, H, ids, weights)
        batch, code = self._rows(X, ids)
        _check_out(dY, (batch, self.n_out), torch.float32, self.device, "dY")
        _check_out(H, (batch, self.rank), torch.float32, self.device, "H")
        dX = self._f32(batch, self.n_in)
        dA = dB = None
        if weights:
            dA = self._f32(self.count, self.rank, self.n_in)
            dB = self._f32(self.count, self.n_out, self.rank)
        wt, launch = None, _raw_stream(self._index)
        if self._wt is not None and [w._version for w in self._keep[0]] == self._versions:
            wt = self._wt.data_ptr()
            if launch != self._wt_stream:              # the handle may go before the kernels are done
                self._wt.record_stream(torch.cuda.current_stream(self._index))
        ws, size, _keep = self._workspace("ks_chain_adapter_backward_workspace_size", batch, code, int(wt is not None))
        _raise(self._lib.ks_chain_adapter_backward(
            self._p, self._n, self._w, wt, self._ad, ids.data_ptr(), dY.data_ptr(), X.data_ptr(), H.data_ptr(),
            dX.data_ptr(), _ptr(dA), _ptr(dB), batch, code, ws, size, launch),
            "ks_chain_adapter_backward", True)
        return dX, dA, dB


def _check_out(t, shape, dtype, device, name):
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.device != device:
        raise ValueError("%s must be %s %s on %s" % (name, tuple(shape), dtype, device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _adapters(A, B, scale, n_in, n_out):
    import torch
    for t, name in ((A, "A"), (B, "B"), (scale, "scale")):
        _check_tensor(t, name)
    if A.dim() != 3 or B.dim() != 3 or tuple(B.shape) != (A.shape[0], n_out, A.shape[1]) or A.shape[2] != n_in:
        raise ValueError("A must be (adapters, rank, %d) and B (adapters, %d, rank)" % (n_in, n_out))
    if tuple(scale.shape) != (A.shape[0],) or scale.dtype != torch.float32:
        raise ValueError("scale must be (%d,) fp32" % A.shape[0])
    if A.dtype != B.dtype:
        raise TypeError("A and B must have one type")
    return ks_adapters_t(A.data_ptr(), B.data_ptr(), scale.data_ptr(), n_in, n_out, A.shape[1], A.shape[0])


def adapter_matmul(X, A, B, scale, ids, out, keep=False, stream=None):
    """out (batch, n_out) fp32 += H B^T for any projection's output; returns
    out, or (out, H) with keep=True."""
    import torch
    for t, name in ((X, "X"), (ids, "ids"), (out, "out")):
        _check_tensor(t, name)
    if X.dim() != 2 or out.dim() != 2 or out.shape[0] != X.shape[0] or out.dtype != torch.float32:
        raise ValueError("X must be (batch, n_in) and out (batch, n_out) fp32")
    if ids.dtype != torch.int32 or tuple(ids.shape) != (X.shape[0],):
        raise ValueError("ids must be (batch,) int32")
    if stream is not None:
        return _on_stream(stream, X.device, adapter_matmul, X, A, B, scale, ids, out, keep)
    ad = _adapters(A, B, scale, X.shape[1], out.shape[1])
    H = torch.empty((X.shape[0], ad.rank), dtype=torch.float32, device=X.device)
    size = ctypes.c_size_t(0)
    _raise(load().ks_adapter_workspace_size(ad, X.shape[0], size), "ks_adapter_workspace_size", True)
    ws = torch.empty(size.value, dtype=torch.uint8, device=X.device) if size.value else None
    _raise(load().ks_adapter_matmul(ad, _ptr(ids), _ptr(X), _ptr(out), _ptr(H), X.shape[0],
                                    dtype_code(X.dtype, A.dtype), _ptr(ws), size.value, _stream(None, X)),
           "ks_adapter_matmul", True)
    _wrote(out)
    return (out, H) if keep else out


def adapter_backward(dY, X, H, A, B, scale, ids, dX=None, stream=None):
    """(dA, dB) fp32 of adapter_matmul; dX (batch, n_in) fp32, if given, is
    added to."""
    import torch
    for t, name in ((dY, "dY"), (X, "X"), (H, "H"), (ids, "ids")):
        _check_tensor(t, name)
    if X.dim() != 2 or dY.dim() != 2 or dY.shape[0] != X.shape[0] or dY.dtype != torch.float32:
        raise ValueError("X must be (batch, n_in) and dY (batch, n_out) fp32")
    if ids.dtype != torch.int32 or tuple(ids.shape) != (X.shape[0],):
        raise ValueError("ids must be (batch,) int32")
    if stream is not None:
        return _on_stream(stream, X.device, adapter_backward, dY, X, H, A, B, scale, ids, dX)
    ad = _adapters(A, B, scale, X.shape[1], dY.shape[1])
    _check_out(H, (X.shape[0], ad.rank), torch.float32, X.device, "H")
    if dX is not None:
        _check_out(dX, tuple(X.shape), torch.float32, X.device, "dX")
    dA = torch.empty(tuple(A.shape), dtype=torch.float32, device=X.device)
    dB = torch.empty(tuple(B.shape), dtype=torch.float32, device=X.device)
    size = ctypes.c_size_t(0)
    _raise(load().ks_adapter_backward_workspace_size(ad, X.shape[0], size), "ks_adapter_backward_workspace_size", True)
    ws = torch.empty(max(size.value, 1), dtype=torch.uint8, device=X.device)
    _raise(load().ks_adapter_backward(ad, _ptr(ids), _ptr(dY), _ptr(X), _ptr(H), _ptr(dX), _ptr(dA), _ptr(dB),
                                      X.shape[0], dtype_code(X.dtype, A.dtype), _ptr(ws), size.value,
                                      _stream(None, X)), "ks_adapter_backward", True)
    if dX is not None:
        _wrote(dX)
    return dA, dB


# ---------------------------------------------------------------- preference loss

def _elem(dtype, name) -> int:
    import torch
    if dtype == torch.float32:
        return ELEM_F32
    if dtype == torch.bfloat16:
        return ELEM_BF16
    raise TypeError("%s must be fp32 or bf16, not %s" % (name, dtype))


def _layout(x, name):
    """(sequence stride, row stride) of (S, T, V) values with contiguous rows."""
    S, T, V = x.shape
    seq, row, one = x.stride()
    if V > 1 and one != 1:
        raise ValueError("the last dimension of %s must be contiguous" % name)
    # strides of dimensions with at most one entry say nothing
    if T <= 1:
        row = max(V, 1)
    if S <= 1:
        seq = max((T - 1) * row + V, 0)
    return seq, row


def _rows_stride(t, name):
    S, T = t.shape
    seq, one = t.stride()
    if T > 1 and one != 1:
        raise ValueError("the rows of %s must be contiguous" % name)
    return seq if S > 1 else T


def _logits(x, labels) -> ks_logits_t:
    import torch
    if x.dim() != 3 or labels.shape != x.shape[:2]:
        raise ValueError("logits must be (sequences, tokens, vocab) and labels (sequences, tokens)")
    if labels.dtype != torch.int64:
        raise TypeError("labels must be int64")
    if not x.is_cuda or labels.get_device() != x.get_device():
        raise ValueError("logits and labels must be device tensors on one device")
    seq, row = _layout(x, "logits")
    return ks_logits_t(x.data_ptr(), labels.data_ptr(), seq, row, _rows_stride(labels, "labels"), *x.shape,
                       _elem(x.dtype, "logits"), 0)


def sequence_logp(logits, labels, stream=None):
    """(total, tokens): log probabilities of the labels, summed over each
    sequence and for each token. logits (S, T, V) fp32 or bf16 with any row
    strides; labels (S, T) int64, negative where masked."""
    import torch
    x = _logits(logits, labels)
    if stream is not None:
        return _on_stream(stream, logits.device, sequence_logp, logits, labels)
    tokens = torch.empty((x.sequences, x.tokens), dtype=torch.float32, device=logits.device)
    total = torch.empty((x.sequences,), dtype=torch.float32, device=logits.device)
    _raise(load().ks_sequence_logp(x, tokens.data_ptr(), total.data_ptr(), None,
                                   _raw_stream(logits.get_device())), "ks_sequence_logp", True)
    return total, tokens


def _preference_forward(logits, labels, ref, beta, smoothing, dlogits=None):
    """(loss, rewards, tokens, scratch): scratch holds d loss / d total, then
    the rows' statistics."""
    import torch
    x = _logits(logits, labels)
    if ref.dtype != torch.float32 or ref.shape != labels.shape or ref.get_device() != logits.get_device():
        raise ValueError("ref must be (sequences, tokens) fp32 on the logits' device")
    d_seq = d_row = 0
    if dlogits is not None:
        if dlogits.shape != logits.shape or dlogits.dtype != logits.dtype \
                or dlogits.get_device() != logits.get_device():
            raise ValueError("dlogits must have the logits' shape, type and device")
        d_seq, d_row = _layout(dlogits, "dlogits")
    S, T = x.sequences, x.tokens
    # memory of their own: as views of one buffer the results could not be changed
    # in place under autograd, and would keep each other alive
    loss = torch.empty((), dtype=torch.float32, device=logits.device)
    f32 = loss.new_empty
    rewards, tokens, scratch = f32(S), f32(S, T), f32(S + 2 * S * T)
    at = scratch.data_ptr()
    _raise(load().ks_preference_loss(x, ref.data_ptr(), _rows_stride(ref, "ref"), float(beta), float(smoothing),
                                     loss.data_ptr(), rewards.data_ptr(), tokens.data_ptr(), at, at + 4 * S,
                                     _ptr(dlogits), d_seq, d_row, _raw_stream(logits.get_device())),
           "ks_preference_loss", True)
    return loss, rewards, tokens, scratch


def preference_loss(logits, labels, ref, beta=0.1, smoothing=0.0, dlogits=None, stream=None):
    """(loss, rewards, tokens, dlogits) of the paired preference loss: sequences
    0..P-1 of the logits (2P, T, V) are the chosen answers, P..2P-1 the rejected
    ones, ref (2P, T) fp32 the reference model's token log probabilities.
    dlogits may be given (the logits themselves too: then it replaces them)."""
    import torch
    if stream is not None:
        _logits(logits, labels)
        return _on_stream(stream, logits.device, preference_loss, logits, labels, ref, beta, smoothing, dlogits)
    given = dlogits is not None
    if not given:
        dlogits = torch.empty_like(logits, memory_format=torch.contiguous_format)
    loss, rewards, tokens, _ = _preference_forward(logits, labels, ref, beta, smoothing, dlogits)
    if given:
        _wrote(dlogits)
    return loss, rewards, tokens, dlogits


def _preference_backward(logits, labels, scratch, upstream):
    import torch
    dlogits = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    x = _logits(logits, labels)
    d_seq, d_row = _layout(dlogits, "dlogits")
    at = scratch.data_ptr()
    _raise(load().ks_preference_backward(x, at + 4 * x.sequences, at, _ptr(upstream), dlogits.data_ptr(), d_seq, d_row,
                                         _raw_stream(logits.get_device())), "ks_preference_backward", True)
    return dlogits


# ---------------------------------------------------------------- optimizer

ADAMW_BLOCK = 256   # values that share a scale in 8 bits
_dtype_of, _base_of = operator.attrgetter("dtype"), operator.attrgetter("_base")


class AdamW:
    """One AdamW step over many tensors. The handle keeps the tensors it was
    given (params, grads and the moments ms, vs, changed in place) and their
    addresses. Moments are fp32, or with `scales` int8 (ms) and uint8 (vs) with
    scales[i] of shape (ceil(n / 256), 2), fp32."""

    def __init__(self, params, grads, ms, vs, scales=None):
        import torch
        n = len(params)
        if not (len(grads) == len(ms) == len(vs) == n) or (scales is not None and len(scales) != n):
            raise ValueError("params, grads, ms, vs and scales must have one entry a tensor")
        self.bits = 32 if scales is None else 8
        types = (torch.float32, torch.float32) if scales is None else (torch.int8, torch.uint8)
        self._n = n
        self.device = params[0].device if n else None
        T = torch.Tensor
        self._sizes = list(map(T.numel, params))
        index = self.device.index if n else None
        sets = [(params, "params"), (grads, "grads"), (ms, "ms"), (vs, "vs")]
        for ts, name in sets:
            if list(map(T.numel, ts)) != self._sizes:
                raise ValueError("%s must have their parameters' sizes" % name)
        if scales is not None:
            sets.append((scales, "scales"))
            if [t.shape for t in scales] != [(-(-size // ADAMW_BLOCK), 2) for size in self._sizes] \
                    or any(t.dtype is not torch.float32 for t in scales):
                raise ValueError("scales must be (ceil(n / %d), 2) fp32" % ADAMW_BLOCK)
        for ts, name in sets:
            if not all(t.is_cuda for t in ts) or not all(map(T.is_contiguous, ts)) \
                    or any(d != index for d in map(T.get_device, ts)):
                raise ValueError("%s must be contiguous, on one device" % name)
        if any(t.dtype is not types[0] for t in ms) or any(t.dtype is not types[1] for t in vs):
            raise TypeError("moments must be %s and %s" % types)
        at = [list(map(T.data_ptr, ts)) for ts in (params, grads, ms, vs)]
        at.append(list(map(T.data_ptr, scales)) if scales is not None else [None] * n)
        for ts, name in ((params, "params"), (grads, "grads")):
            codes = {t: _elem(t, name) for t in set(map(_dtype_of, ts))}
            at.append([codes[t] for t in map(_dtype_of, ts)])
        self._t = (ks_adamw_tensor_t * max(n, 1))(*zip(*at[:5], self._sizes, *at[5:]))
        spans = []
        for ts, addr in ((params, at[0]), (ms, at[2]), (vs, at[3]), (scales or [], at[4])):
            spans += [(a, a + b) for a, b in zip(addr, [t.nbytes for t in ts]) if b]
        spans.sort()
        if any(b[0] < a[1] for a, b in zip(spans, spans[1:])):
            raise ValueError("parameters and moments must not share memory")
        self._keep = (list(params), list(grads), list(ms), list(vs), list(scales or ()))
        self._written = self._counters(params, ms, vs, scales or ())
        self._lib = load()
        size = ctypes.c_size_t(0)
        _raise(self._lib.ks_grad_norm_workspace_size(self._t, n, size), "ks_grad_norm_workspace_size", True)
        self._ws_bytes = size.value

    @staticmethod
    def _counters(*sets):
        """Tensors that hold the version counters of all of these: views of one
        buffer share its counter."""
        out = []
        for ts in sets:
            if ts and ts[0]._base is not None:
                bases = set(map(_base_of, ts))
                ts = [t for t in ts if t._base is None] if None in bases else []
                out += bases - {None}
            out += ts
        return out

    def _check_scalar(self, t, name):
        import torch
        if not isinstance(t, torch.Tensor) or t.numel() != 1 or t.dtype is not torch.float32 or t.device != self.device:
            raise ValueError("%s must be one fp32 value on %s" % (name, self.device))

    def grad_norm(self, out=None, stream=None):
        """The 2-norm over all gradients, a device scalar."""
        import torch
        if stream is not None:
            return _on_stream(stream, self.device, self.grad_norm, out)
        given = out is not None
        if not given:
            out = torch.empty((), dtype=torch.float32, device=self.device)
        else:
            self._check_scalar(out, "out")
        ws = torch.empty(max(self._ws_bytes, 1), dtype=torch.uint8, device=self.device)
        _raise(self._lib.ks_grad_norm(self._t, self._n, out.data_ptr(), ws.data_ptr(), self._ws_bytes,
                                      _raw_stream(self.device.index)), "ks_grad_norm", True)
        if given:
            _wrote(out)
        return out

    def step(self, step, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, max_norm=None, norm=None, seed=0,
             stream=None):
        """The step number `step` (from 1). max_norm: scale the gradients to at
        most that norm, `norm` (a device scalar) or grad_norm(); a norm that is
        not finite leaves everything as it was. Returns the norm used, or
        None."""
        if self._n == 0:
            return norm
        if max_norm is not None and not max_norm > 0:
            raise ValueError("max_norm must be positive")
        if norm is not None:
            self._check_scalar(norm, "norm")
        if stream is not None:
            return _on_stream(stream, self.device, self.step, step, lr, betas, eps, weight_decay, max_norm, norm, seed)
        if max_norm is not None and norm is None:
            norm = self.grad_norm()
        o = ks_adamw_options_t(float(lr), float(betas[0]), float(betas[1]), float(eps), float(weight_decay),
                               float(max_norm or 0.0), int(step), int(seed) & 0xFFFFFFFF, self.bits)
        _raise(self._lib.ks_adamw_step(self._t, self._n, o, _ptr(norm) if max_norm is not None else None,
                                       _raw_stream(self.device.index)), "ks_adamw_step", True)
        _wrote(self._written)
        return norm

    def state_values(self, ms_out, vs_out, stream=None):
        """The values that 8-bit moments stand for, into fp32 tensors."""
        import torch
        if stream is not None:
            return _on_stream(stream, self.device, self.state_values, ms_out, vs_out)
        if self.bits != 8:
            raise ValueError("32-bit moments are their own values")
        if len(ms_out) != self._n or len(vs_out) != self._n:
            raise ValueError("one output a tensor")
        if self._n == 0:
            return
        T, index, ptrs = torch.Tensor, self.device.index, []
        for outs in (ms_out, vs_out):
            if list(map(T.numel, outs)) != self._sizes or set(map(_dtype_of, outs)) != {torch.float32}:
                raise ValueError("outputs must be fp32 of their parameter's size")
            if set(map(T.get_device, outs)) != {index} or not all(map(T.is_contiguous, outs)):
                raise ValueError("outputs must be contiguous, on the parameters' device")
            ptrs.append((ctypes.c_void_p * self._n).from_buffer(array.array("Q", map(T.data_ptr, outs))))
        _raise(self._lib.ks_adamw_state_values(self._t, self._n, *ptrs, _raw_stream(index)),
               "ks_adamw_state_values", True)
        _wrote([*ms_out, *vs_out])
