"""ctypes binding of libqk.so with the same names as the C ABI (include/qk.h).

Argument marshalling only: pointers, sizes, dtype codes and streams are
converted and passed through; the operators themselves run in the CUDA
kernels of libqk.so.  A non-OK status raises QkError.  There is no fallback:
if the library is missing every call raises.

The ``softmax_fwd`` / ``rmsnorm_fwd`` / ``layernorm_fwd`` / ``xent_fwd`` helpers take
and return CUDA tensors (they allocate the outputs with PyTorch and then call
the C entry points), and so do ``add_rmsnorm_fwd`` / ``add_rmsnorm_bwd`` /
``rmsnorm_quant_fwd`` / ``linear_xent_fwd`` / ``linear_xent_bwd``, which allocate
their workspaces too.  A helper runs on torch's current stream, or on the
``stream`` it is given, which has to have waited for the inputs.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(_HERE, "_lib", "libqk.so")

QK_F32, QK_BF16 = 0, 1
QK_OP_SOFTMAX, QK_OP_RMSNORM, QK_OP_XENT = 0, 1, 2
QK_OP_SOFTMAX_BWD, QK_OP_RMSNORM_BWD, QK_OP_XENT_BWD = 3, 4, 5
QK_OP_LAYERNORM = 6
QK_OK = 0
QK_ERR_INVALID_ARG = 1
QK_ERR_UNSUPPORTED = 2
QK_ERR_MISALIGNED = 3
QK_ERR_LAUNCH = 4
QK_ERR_TIMEOUT = 5
QK_ERR_NO_DEVICE = 6
QK_E4M3, QK_INT8 = 0, 1

_EXPORTS = (
    "qk_softmax_fwd", "qk_rmsnorm_fwd", "qk_xent_fwd", "qk_status_string",
    "qk_get_device_status", "qk_max_row_elements", "qk_get_plan",
    "qk_set_plan_override", "qk_test_wait_timeout", "qk_softmax_bwd", "qk_rmsnorm_bwd",
    "qk_rmsnorm_bwd_workspace_size", "qk_xent_bwd", "qk_rmsnorm_bwd_noalloc",
    "qk_xent_fwd_ex", "qk_xent_bwd_ex", "qk_layernorm_fwd", "qk_add_rmsnorm_fwd",
    "qk_add_rmsnorm_bwd", "qk_add_rmsnorm_bwd_workspace_size", "qk_rmsnorm_quant_fwd",
    "qk_linear_xent_fwd", "qk_linear_xent_fwd_workspace_size", "qk_linear_xent_bwd",
    "qk_linear_xent_bwd_workspace_size",
)


class QkError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {qk_status_string(status)} (status {status})")


class qk_xent_options(ctypes.Structure):
    _fields_ = [("has_ignore_index", ctypes.c_int32), ("z_loss", ctypes.c_float),
                ("ignore_index", ctypes.c_int64)]


class qk_plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "path", "threads", "row_threads", "vec_per_thread", "cluster", "slots", "chunks",
        "ctas_per_sm", "grid", "smem_bytes")]

    def as_dict(self) -> dict:
        return {n: getattr(self, n) for n, _ in self._fields_}


_lock = threading.Lock()
_lib = None


def load_library(path: str = LIBRARY):
    """Load libqk.so (once) and declare its signatures; raises if it is missing."""
    global _lib
    lib = _lib
    if lib is not None:  # every call after the first: no lock
        return lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build the CUDA library first "
                "(python -m memory_bound_row_rmsnorm_gb300.build)")
        lib = ctypes.CDLL(path)
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        fp = ctypes.POINTER(ctypes.c_float)
        lib.qk_softmax_fwd.argtypes = [vp, vp, i64, i64, i32, vp]
        lib.qk_rmsnorm_fwd.argtypes = [vp, vp, vp, vp, i64, i64, ctypes.c_float, i32, vp]
        lib.qk_xent_fwd.argtypes = [vp, vp, vp, vp, i64, i64, i32, vp]
        lib.qk_status_string.argtypes = [i32]
        lib.qk_status_string.restype = ctypes.c_char_p
        lib.qk_get_device_status.argtypes = [vp]
        lib.qk_max_row_elements.argtypes = [i32, i32]
        lib.qk_max_row_elements.restype = i64
        lib.qk_get_plan.argtypes = [i32, i32, i64, i64, ctypes.POINTER(qk_plan)]
        lib.qk_set_plan_override.argtypes = [i32, i32, ctypes.POINTER(qk_plan)]
        lib.qk_test_wait_timeout.argtypes = [ctypes.c_uint64, vp]
        lib.qk_softmax_bwd.argtypes = [vp, vp, vp, i64, i64, i32, vp]
        lib.qk_rmsnorm_bwd_workspace_size.argtypes = [i64, i64, i32, ctypes.POINTER(ctypes.c_size_t)]
        lib.qk_rmsnorm_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, i64, i64, i32, vp]
        lib.qk_xent_bwd.argtypes = [vp, vp, vp, vp, vp, i64, i64, i32, vp]
        lib.qk_rmsnorm_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i32, vp]
        op = ctypes.POINTER(qk_xent_options)
        lib.qk_xent_fwd_ex.argtypes = [vp, vp, vp, vp, vp, i64, i64, i32, op, vp]
        lib.qk_xent_bwd_ex.argtypes = [vp, vp, vp, vp, vp, i64, i64, i32, op, vp]
        lib.qk_layernorm_fwd.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, ctypes.c_float, i32, vp]
        sp, f32 = ctypes.POINTER(ctypes.c_size_t), ctypes.c_float
        lib.qk_add_rmsnorm_fwd.argtypes = [vp] * 6 + [i64, i64, f32, i32, vp]
        lib.qk_add_rmsnorm_bwd_workspace_size.argtypes = [i64, i64, i32, sp]
        lib.qk_add_rmsnorm_bwd.argtypes = [vp] * 8 + [ctypes.c_size_t, i64, i64, i32, vp]
        lib.qk_rmsnorm_quant_fwd.argtypes = [vp] * 7 + [i64, i64, f32, i64, i32, i32, vp]
        lib.qk_linear_xent_fwd_workspace_size.argtypes = [i64, i64, i64, i32, sp]
        lib.qk_linear_xent_fwd.argtypes = [vp] * 7 + [ctypes.c_size_t, i64, i64, i64, i32, op, vp]
        lib.qk_linear_xent_bwd_workspace_size.argtypes = [i64, i64, i64, i32, sp]
        lib.qk_linear_xent_bwd.argtypes = [vp] * 8 + [ctypes.c_size_t, i64, i64, i64, i32, op, vp]
        for name in ("qk_softmax_fwd", "qk_rmsnorm_fwd", "qk_xent_fwd", "qk_get_device_status",
                     "qk_get_plan", "qk_set_plan_override", "qk_test_wait_timeout",
                     "qk_softmax_bwd", "qk_rmsnorm_bwd_workspace_size", "qk_rmsnorm_bwd",
                     "qk_xent_bwd", "qk_rmsnorm_bwd_noalloc", "qk_xent_fwd_ex", "qk_xent_bwd_ex",
                     "qk_layernorm_fwd", "qk_add_rmsnorm_fwd", "qk_add_rmsnorm_bwd_workspace_size",
                     "qk_add_rmsnorm_bwd", "qk_rmsnorm_quant_fwd", "qk_linear_xent_fwd_workspace_size",
                     "qk_linear_xent_fwd", "qk_linear_xent_bwd_workspace_size", "qk_linear_xent_bwd"):
            getattr(lib, name).restype = i32
        del fp
        _lib = lib
        return lib


def _ptr(p) -> int | None:
    """A device pointer from an int, None, or anything with data_ptr()."""
    if p is None:
        return None
    if hasattr(p, "data_ptr"):
        return p.data_ptr()
    return int(p)


def _stream(s) -> int | None:
    """A cudaStream_t from an int, a torch.cuda.Stream, or None (torch's current stream)."""
    if s is None:
        import sys
        torch = sys.modules.get("torch")
        if torch is not None and torch.cuda.is_available() and torch.cuda.is_initialized():
            return torch.cuda.current_stream().cuda_stream or None
        return None
    if hasattr(s, "cuda_stream"):
        return s.cuda_stream or None
    return int(s) or None


def _check(st: int, where: str) -> None:
    if st != QK_OK:
        raise QkError(st, where)


# --- the C entry points, same names -----------------------------------------
def qk_softmax_fwd(x, y, M: int, N: int, dtype: int, stream=None) -> None:
    _check(load_library().qk_softmax_fwd(_ptr(x), _ptr(y), M, N, dtype, _stream(stream)),
           "qk_softmax_fwd")


def qk_rmsnorm_fwd(x, w, y, rstd, M: int, N: int, eps: float, dtype: int, stream=None) -> None:
    _check(load_library().qk_rmsnorm_fwd(_ptr(x), _ptr(w), _ptr(y), _ptr(rstd), M, N, eps, dtype,
                                         _stream(stream)), "qk_rmsnorm_fwd")


def qk_layernorm_fwd(x, w, b, y, mean, rstd, M: int, N: int, eps: float, dtype: int,
                     stream=None) -> None:
    _check(load_library().qk_layernorm_fwd(_ptr(x), _ptr(w), _ptr(b), _ptr(y), _ptr(mean),
                                           _ptr(rstd), M, N, eps, dtype, _stream(stream)),
           "qk_layernorm_fwd")


def qk_xent_fwd(logits, targets, loss, lse, M: int, N: int, dtype: int, stream=None) -> None:
    _check(load_library().qk_xent_fwd(_ptr(logits), _ptr(targets), _ptr(loss), _ptr(lse), M, N,
                                      dtype, _stream(stream)), "qk_xent_fwd")


def qk_softmax_bwd(y, dy, dx, M: int, N: int, dtype: int, stream=None) -> None:
    _check(load_library().qk_softmax_bwd(_ptr(y), _ptr(dy), _ptr(dx), M, N, dtype, _stream(stream)),
           "qk_softmax_bwd")


def qk_rmsnorm_bwd_workspace_size(M: int, N: int, dtype: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().qk_rmsnorm_bwd_workspace_size(M, N, dtype, ctypes.byref(n)),
           "qk_rmsnorm_bwd_workspace_size")
    return n.value


def qk_rmsnorm_bwd(x, w, rstd, dy, dx, dw, workspace, workspace_bytes: int, M: int, N: int,
                   dtype: int, stream=None) -> None:
    _check(load_library().qk_rmsnorm_bwd(_ptr(x), _ptr(w), _ptr(rstd), _ptr(dy), _ptr(dx), _ptr(dw),
                                         _ptr(workspace), int(workspace_bytes), M, N, dtype,
                                         _stream(stream)), "qk_rmsnorm_bwd")


def qk_rmsnorm_bwd_noalloc(x, w, rstd, dy, dx, dw, M: int, N: int, dtype: int, stream=None) -> None:
    """qk_rmsnorm_bwd with the workspace taken from the library's fixed device
    array (for callers that cannot allocate device memory)."""
    _check(load_library().qk_rmsnorm_bwd_noalloc(_ptr(x), _ptr(w), _ptr(rstd), _ptr(dy), _ptr(dx),
                                                 _ptr(dw), M, N, dtype, _stream(stream)),
           "qk_rmsnorm_bwd_noalloc")


def qk_xent_bwd(logits, targets, lse, dloss, dlogits, M: int, N: int, dtype: int, stream=None) -> None:
    _check(load_library().qk_xent_bwd(_ptr(logits), _ptr(targets), _ptr(lse), _ptr(dloss),
                                      _ptr(dlogits), M, N, dtype, _stream(stream)), "qk_xent_bwd")


def _options(ignore_index, z_loss):
    if ignore_index is None and not z_loss:
        return None
    return ctypes.byref(qk_xent_options(
        0 if ignore_index is None else 1, float(z_loss), 0 if ignore_index is None else int(ignore_index)))


def qk_xent_fwd_ex(logits, targets, loss, lse, mean_loss, M: int, N: int, dtype: int,
                   ignore_index=None, z_loss: float = 0.0, stream=None) -> None:
    _check(load_library().qk_xent_fwd_ex(_ptr(logits), _ptr(targets), _ptr(loss), _ptr(lse),
                                         _ptr(mean_loss), M, N, dtype, _options(ignore_index, z_loss),
                                         _stream(stream)), "qk_xent_fwd_ex")


def qk_xent_bwd_ex(logits, targets, lse, dloss, dlogits, M: int, N: int, dtype: int,
                   ignore_index=None, z_loss: float = 0.0, stream=None) -> None:
    _check(load_library().qk_xent_bwd_ex(_ptr(logits), _ptr(targets), _ptr(lse), _ptr(dloss),
                                         _ptr(dlogits), M, N, dtype, _options(ignore_index, z_loss),
                                         _stream(stream)), "qk_xent_bwd_ex")


def qk_add_rmsnorm_fwd(x, residual, w, y, h, rstd, M: int, N: int, eps: float, dtype: int,
                       stream=None) -> None:
    _check(load_library().qk_add_rmsnorm_fwd(_ptr(x), _ptr(residual), _ptr(w), _ptr(y), _ptr(h),
                                             _ptr(rstd), M, N, eps, dtype, _stream(stream)),
           "qk_add_rmsnorm_fwd")


def qk_add_rmsnorm_bwd_workspace_size(M: int, N: int, dtype: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().qk_add_rmsnorm_bwd_workspace_size(M, N, dtype, ctypes.byref(n)),
           "qk_add_rmsnorm_bwd_workspace_size")
    return n.value


def qk_add_rmsnorm_bwd(h, w, rstd, dy, dh, dx, dw, workspace, workspace_bytes: int, M: int, N: int,
                       dtype: int, stream=None) -> None:
    _check(load_library().qk_add_rmsnorm_bwd(_ptr(h), _ptr(w), _ptr(rstd), _ptr(dy), _ptr(dh), _ptr(dx),
                                             _ptr(dw), _ptr(workspace), int(workspace_bytes), M, N, dtype,
                                             _stream(stream)), "qk_add_rmsnorm_bwd")


def qk_rmsnorm_quant_fwd(x, residual, w, q, scale, h, rstd, M: int, N: int, eps: float, group: int,
                         dtype: int, qtype: int, stream=None) -> None:
    _check(load_library().qk_rmsnorm_quant_fwd(_ptr(x), _ptr(residual), _ptr(w), _ptr(q), _ptr(scale),
                                               _ptr(h), _ptr(rstd), M, N, eps, group, dtype, qtype,
                                               _stream(stream)), "qk_rmsnorm_quant_fwd")


def qk_linear_xent_fwd_workspace_size(M: int, V: int, K: int, dtype: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().qk_linear_xent_fwd_workspace_size(M, V, K, dtype, ctypes.byref(n)),
           "qk_linear_xent_fwd_workspace_size")
    return n.value


def qk_linear_xent_fwd(h, w, targets, loss, lse, mean_loss, workspace, workspace_bytes: int, M: int,
                       V: int, K: int, dtype: int, ignore_index=None, z_loss: float = 0.0,
                       stream=None) -> None:
    _check(load_library().qk_linear_xent_fwd(_ptr(h), _ptr(w), _ptr(targets), _ptr(loss), _ptr(lse),
                                             _ptr(mean_loss), _ptr(workspace), int(workspace_bytes), M, V,
                                             K, dtype, _options(ignore_index, z_loss), _stream(stream)),
           "qk_linear_xent_fwd")


def qk_linear_xent_bwd_workspace_size(M: int, V: int, K: int, dtype: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().qk_linear_xent_bwd_workspace_size(M, V, K, dtype, ctypes.byref(n)),
           "qk_linear_xent_bwd_workspace_size")
    return n.value


def qk_linear_xent_bwd(h, w, targets, lse, dloss, dh, dw, workspace, workspace_bytes: int, M: int, V: int,
                       K: int, dtype: int, ignore_index=None, z_loss: float = 0.0, stream=None) -> None:
    _check(load_library().qk_linear_xent_bwd(_ptr(h), _ptr(w), _ptr(targets), _ptr(lse), _ptr(dloss),
                                             _ptr(dh), _ptr(dw), _ptr(workspace), int(workspace_bytes), M,
                                             V, K, dtype, _options(ignore_index, z_loss), _stream(stream)),
           "qk_linear_xent_bwd")


def qk_status_string(status: int) -> str:
    return load_library().qk_status_string(status).decode()


def qk_get_device_status(stream=None) -> int:
    """Returns (does not raise) the device status word, clearing it."""
    return load_library().qk_get_device_status(_stream(stream))


def qk_max_row_elements(op: int, dtype: int) -> int:
    return load_library().qk_max_row_elements(op, dtype)


def qk_get_plan(op: int, dtype: int, M: int, N: int) -> dict:
    p = qk_plan()
    _check(load_library().qk_get_plan(op, dtype, M, N, ctypes.byref(p)), "qk_get_plan")
    return p.as_dict()


def qk_set_plan_override(op: int, dtype: int, plan: dict | None) -> None:
    if plan is None:
        _check(load_library().qk_set_plan_override(op, dtype, None), "qk_set_plan_override")
        return
    p = qk_plan(**{k: int(v) for k, v in plan.items() if k in dict(qk_plan._fields_)})
    _check(load_library().qk_set_plan_override(op, dtype, ctypes.byref(p)), "qk_set_plan_override")


def qk_test_wait_timeout(timeout_ns: int, stream=None) -> None:
    _check(load_library().qk_test_wait_timeout(int(timeout_ns), _stream(stream)),
           "qk_test_wait_timeout")


# --- tensor helpers ----------------------------------------------------------
def _on(stream, helper, *args):
    """helper(*args) on `stream` (a torch.cuda.Stream or a cudaStream_t).  Torch
    hands freed memory out again at once, in the order of the stream that it
    belongs to.  So `stream` is torch's current one meanwhile, and what the
    helper allocates is that stream's: memory of the caller's stream may have
    work on that stream before it, for which `stream` does not wait.  The tensors
    that cross from one stream to the other are known to the allocator as used on
    both, so that their memory is not handed out while either still reads them.
    The inputs have to be ready: `stream` waits for nothing here."""
    import torch
    if not args[0].is_cuda:
        raise ValueError("expected a CUDA tensor")
    dev = args[0].get_device()
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(getattr(stream, "cuda_stream", stream))
        # 0 and 1 name the legacy default stream, which torch's default stream is
        stream = torch.cuda.ExternalStream(handle, device=dev) if handle > 1 else torch.cuda.default_stream(dev)
    if stream.device_index != dev:
        raise ValueError(f"the tensors are on cuda:{dev}, the stream is of device {stream.device_index}")
    caller = torch.cuda.current_stream(dev)
    with torch.cuda.stream(stream):
        out = helper(*args)
    if stream.cuda_stream != caller.cuda_stream:
        for t in args:
            if hasattr(t, "record_stream"):
                t.record_stream(stream)
        for t in out if isinstance(out, tuple) else (out,):
            if t is not None:
                t.record_stream(caller)
    return out


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return QK_F32
    if t.dtype == torch.bfloat16:
        return QK_BF16
    raise TypeError(f"unsupported dtype {t.dtype}: float32 or bfloat16 expected")


def _rows(x):
    if not x.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not x.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    N = x.shape[-1] if x.dim() > 0 else 1
    return x.numel() // max(N, 1), N


def softmax_fwd(x, out=None, stream=None):
    """Row-wise softmax over the last dimension of a CUDA tensor."""
    if stream is not None:
        return _on(stream, softmax_fwd, x, out)
    import torch
    M, N = _rows(x)
    y = torch.empty_like(x) if out is None else out
    qk_softmax_fwd(x, y, M, N, _dtype_code(x))
    return y


def rmsnorm_fwd(x, w, eps: float = 1e-6, out=None, want_rstd: bool = True, stream=None):
    """RMSNorm over the last dimension; returns (y, rstd) (rstd is None if not wanted)."""
    if stream is not None:
        return _on(stream, rmsnorm_fwd, x, w, eps, out, want_rstd)
    import torch
    M, N = _rows(x)
    if w.dtype != x.dtype or w.numel() != N or not w.is_contiguous():
        raise ValueError("w must be a contiguous [N] tensor of x's dtype")
    y = torch.empty_like(x) if out is None else out
    rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device) if want_rstd else None
    qk_rmsnorm_fwd(x, w, y, rstd, M, N, eps, _dtype_code(x))
    return y, rstd


def layernorm_fwd(x, w, b=None, eps: float = 1e-5, out=None, want_stats: bool = True,
                  stream=None):
    """LayerNorm over the last dimension; returns (y, mean, rstd) (the two
    statistics are None if not wanted).  b may be None (no bias)."""
    if stream is not None:
        return _on(stream, layernorm_fwd, x, w, b, eps, out, want_stats)
    import torch
    M, N = _rows(x)
    for name, t in (("w", w), ("b", b)):
        if t is not None and (t.dtype != x.dtype or t.numel() != N or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous [N] tensor of x's dtype")
    y = torch.empty_like(x) if out is None else out
    mean = rstd = None
    if want_stats:
        mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    qk_layernorm_fwd(x, w, b, y, mean, rstd, M, N, eps, _dtype_code(x))
    return y, mean, rstd


def xent_fwd(logits, targets, want_lse: bool = True, ignore_index=None, z_loss: float = 0.0,
             want_mean: bool = False, stream=None):
    """Per-row cross-entropy; returns (loss, lse) (lse is None if not wanted),
    or (loss, lse, mean) with want_mean."""
    if stream is not None:
        return _on(stream, xent_fwd, logits, targets, want_lse, ignore_index, z_loss, want_mean)
    import torch
    M, N = _rows(logits)
    if targets.dtype != torch.int64 or targets.numel() != M or not targets.is_contiguous():
        raise ValueError("targets must be a contiguous int64 tensor with one entry per row")
    loss = torch.empty(logits.shape[:-1], dtype=torch.float32, device=logits.device)
    lse = torch.empty_like(loss) if want_lse else None
    if ignore_index is None and not z_loss and not want_mean:
        qk_xent_fwd(logits, targets, loss, lse, M, N, _dtype_code(logits))
        return loss, lse
    mean = torch.empty((), dtype=torch.float32, device=logits.device) if want_mean else None
    qk_xent_fwd_ex(logits, targets, loss, lse, mean, M, N, _dtype_code(logits), ignore_index, z_loss)
    return (loss, lse, mean) if want_mean else (loss, lse)


def softmax_bwd(y, dy, out=None, stream=None):
    """Softmax backward over the last dimension: y * (dy - sum(dy * y))."""
    if stream is not None:
        return _on(stream, softmax_bwd, y, dy, out)
    import torch
    M, N = _rows(y)
    dx = torch.empty_like(y) if out is None else out
    qk_softmax_bwd(y, dy, dx, M, N, _dtype_code(y))
    return dx


def rmsnorm_bwd(x, w, rstd, dy, stream=None):
    """RMSNorm backward; returns (dx, dw) with dw in float32.  Allocates the
    workspace with PyTorch (the library itself allocates nothing)."""
    if stream is not None:
        return _on(stream, rmsnorm_bwd, x, w, rstd, dy)
    import torch
    M, N = _rows(x)
    code = _dtype_code(x)
    ws_bytes = qk_rmsnorm_bwd_workspace_size(M, N, code)
    ws = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=x.device)
    dx = torch.empty_like(x)
    dw = torch.empty(N, dtype=torch.float32, device=x.device)
    qk_rmsnorm_bwd(x, w, rstd, dy, dx, dw, ws, ws_bytes, M, N, code)
    return dx, dw


def xent_bwd(logits, targets, lse, dloss=None, ignore_index=None, z_loss: float = 0.0, stream=None):
    """Cross-entropy backward: dloss * ((1 + 2 z lse) softmax(logits) - onehot(targets))."""
    if stream is not None:
        return _on(stream, xent_bwd, logits, targets, lse, dloss, ignore_index, z_loss)
    import torch
    M, N = _rows(logits)
    dx = torch.empty_like(logits)
    qk_xent_bwd_ex(logits, targets, lse, dloss, dx, M, N, _dtype_code(logits), ignore_index, z_loss)
    return dx


# The helpers below serve calls of a few microseconds (a decoding step's norm),
# so their checks are few and cheap: identities, integers, no temporary objects,
# and torch looked up once (_matrix, which every helper calls first, does it).
torch = None


def _matrix(x):
    """(M, N, dtype code, device index) of a contiguous CUDA tensor on the
    current device, where the C entry points launch."""
    global torch
    if torch is None:
        import torch as _torch
        torch = _torch
    dev = x.get_device()
    if dev < 0:
        raise ValueError("expected a CUDA tensor")
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"the tensors are on cuda:{dev}, the current device is cuda:{torch.cuda.current_device()}")
    if not x.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    if x.dtype is torch.bfloat16:
        code = QK_BF16
    elif x.dtype is torch.float32:
        code = QK_F32
    else:
        raise TypeError(f"unsupported dtype {x.dtype}: float32 or bfloat16 expected")
    N = x.shape[-1] if x.dim() > 0 else 1
    return x.numel() // max(N, 1), N, code, dev


def _same(name, t, shape, dtype, dev):
    """t, checked to be a contiguous tensor of that shape, type and device."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")
    return t


def _current_stream(dev):
    """The handle of torch's current stream on device dev."""
    return torch._C._cuda_getCurrentRawStream(dev) or None


@functools.lru_cache(maxsize=512)
def _workspace_bytes(size, dev, *sizes):
    """Bytes that a call of these sizes needs on device dev (`size`: its C function's wrapper)."""
    return size(*sizes)


def add_rmsnorm_fwd(x, residual, w, eps: float = 1e-6, out=None, out_h=None, want_rstd: bool = True,
                    stream=None):
    """h = x + residual and its RMSNorm over the last dimension; returns
    (y, h, rstd) (rstd is None if not wanted).  out and out_h may be x or
    residual (out_h=residual keeps the residual stream in place)."""
    if stream is not None:
        return _on(stream, add_rmsnorm_fwd, x, residual, w, eps, out, out_h, want_rstd)
    M, N, code, dev = _matrix(x)
    shape, dtype = x.shape, x.dtype
    _same("residual", residual, shape, dtype, dev)
    _same("w", w, (N,), dtype, dev)
    y = torch.empty_like(x) if out is None else _same("out", out, shape, dtype, dev)
    h = torch.empty_like(x) if out_h is None else _same("out_h", out_h, shape, dtype, dev)
    rstd = torch.empty(shape[:-1], dtype=torch.float32, device=x.device) if want_rstd else None
    _check(load_library().qk_add_rmsnorm_fwd(
        x.data_ptr(), residual.data_ptr(), w.data_ptr(), y.data_ptr(), h.data_ptr(),
        rstd.data_ptr() if want_rstd else None, M, N, eps, code, _current_stream(dev)), "qk_add_rmsnorm_fwd")
    return y, h, rstd


def add_rmsnorm_bwd(h, w, rstd, dy, dh=None, out=None, stream=None):
    """Backward of add_rmsnorm_fwd; returns (dx, dw): dx is the gradient of x
    and of residual alike, dw is float32.  dh is the gradient that reaches h by
    the residual stream (None: none).  out may be h, dy or dh."""
    if stream is not None:
        return _on(stream, add_rmsnorm_bwd, h, w, rstd, dy, dh, out)
    M, N, code, dev = _matrix(h)
    shape, dtype = h.shape, h.dtype
    _same("w", w, (N,), dtype, dev)
    _same("rstd", rstd, shape[:-1], torch.float32, dev)
    _same("dy", dy, shape, dtype, dev)
    if dh is not None:
        _same("dh", dh, shape, dtype, dev)
    dx = torch.empty_like(h) if out is None else _same("out", out, shape, dtype, dev)
    dw = torch.empty(N, dtype=torch.float32, device=h.device)
    nbytes = _workspace_bytes(qk_add_rmsnorm_bwd_workspace_size, dev, M, N, code)
    ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=h.device)
    _check(load_library().qk_add_rmsnorm_bwd(
        h.data_ptr(), w.data_ptr(), rstd.data_ptr(), dy.data_ptr(), None if dh is None else dh.data_ptr(),
        dx.data_ptr(), dw.data_ptr(), ws.data_ptr(), nbytes, M, N, code, _current_stream(dev)),
        "qk_add_rmsnorm_bwd")
    return dx, dw


def rmsnorm_quant_fwd(x, w, residual=None, eps: float = 1e-6, group: int = 0, qdtype=None, out_h=None,
                      want_h: bool = True, want_rstd: bool = True, stream=None):
    """RMSNorm over the last dimension (of x, or of h = x + residual) with an
    output in 8 bits; returns (q, scale, h, rstd).  q is a qdtype tensor
    (torch.float8_e4m3fn by default, or torch.int8) that stands for
    q * scale; scale has one float32 a row (group 0) or one for each group of
    32, 64 or 128 columns.  h is None without a residual or if not wanted."""
    if stream is not None:
        return _on(stream, rmsnorm_quant_fwd, x, w, residual, eps, group, qdtype, out_h, want_h, want_rstd)
    M, N, code, dev = _matrix(x)
    shape, dtype, device = x.shape, x.dtype, x.device
    if qdtype is None or qdtype is torch.float8_e4m3fn:
        qdtype, qcode = torch.float8_e4m3fn, QK_E4M3
    elif qdtype is torch.int8:
        qcode = QK_INT8
    else:
        raise TypeError(f"unsupported qdtype {qdtype}: torch.float8_e4m3fn or torch.int8 expected")
    if group not in (0, 32, 64, 128):
        raise ValueError("group must be 0 (the whole row), 32, 64 or 128")
    _same("w", w, (N,), dtype, dev)
    h = None
    if residual is not None:
        _same("residual", residual, shape, dtype, dev)
        if out_h is not None:
            h = _same("out_h", out_h, shape, dtype, dev)
        elif want_h:
            h = torch.empty_like(x)
    elif out_h is not None:
        raise ValueError("out_h needs a residual")
    q = torch.empty(shape, dtype=qdtype, device=device)
    scale = torch.empty(shape[:-1] + (-(-N // group) if group else 1,), dtype=torch.float32, device=device)
    rstd = torch.empty(shape[:-1], dtype=torch.float32, device=device) if want_rstd else None
    _check(load_library().qk_rmsnorm_quant_fwd(
        x.data_ptr(), None if residual is None else residual.data_ptr(), w.data_ptr(), q.data_ptr(),
        scale.data_ptr(), None if h is None else h.data_ptr(), rstd.data_ptr() if want_rstd else None, M, N, eps,
        group, code, qcode, _current_stream(dev)), "qk_rmsnorm_quant_fwd")
    return q, scale, h, rstd


def _linear_xent_sizes(h, w, targets):
    M, K, code, dev = _matrix(h)
    if w.dim() != 2:
        raise ValueError("w must have two dimensions, [vocabulary, hidden]")
    V = w.shape[0]
    _same("w", w, (V, K), h.dtype, dev)
    _same("targets", targets, h.shape[:-1], torch.int64, dev)
    return M, V, K, code, dev


def linear_xent_fwd(h, w, targets, want_lse: bool = True, ignore_index=None, z_loss: float = 0.0,
                    want_mean: bool = False, stream=None):
    """Per-row cross-entropy of the logits h @ w.T, which are never stored;
    returns (loss, lse) (lse is None if not wanted), or (loss, lse, mean) with
    want_mean.  Options as in xent_fwd."""
    if stream is not None:
        return _on(stream, linear_xent_fwd, h, w, targets, want_lse, ignore_index, z_loss, want_mean)
    M, V, K, code, dev = _linear_xent_sizes(h, w, targets)
    loss = torch.empty(h.shape[:-1], dtype=torch.float32, device=h.device)
    lse = torch.empty_like(loss) if want_lse else None
    mean = torch.empty((), dtype=torch.float32, device=h.device) if want_mean else None
    nbytes = _workspace_bytes(qk_linear_xent_fwd_workspace_size, dev, M, V, K, code)
    ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=h.device)
    _check(load_library().qk_linear_xent_fwd(
        h.data_ptr(), w.data_ptr(), targets.data_ptr(), loss.data_ptr(), lse.data_ptr() if want_lse else None,
        mean.data_ptr() if want_mean else None, ws.data_ptr(), nbytes, M, V, K, code, _options(ignore_index, z_loss),
        _current_stream(dev)), "qk_linear_xent_fwd")
    return (loss, lse, mean) if want_mean else (loss, lse)


def linear_xent_bwd(h, w, targets, lse, dloss=None, ignore_index=None, z_loss: float = 0.0,
                    want_dh: bool = True, want_dw: bool = True, stream=None):
    """Backward of linear_xent_fwd; returns (dh, dw) (None if not wanted).
    dloss is the float32 gradient of each row's loss (None: 1)."""
    if stream is not None:
        return _on(stream, linear_xent_bwd, h, w, targets, lse, dloss, ignore_index, z_loss, want_dh, want_dw)
    M, V, K, code, dev = _linear_xent_sizes(h, w, targets)
    _same("lse", lse, h.shape[:-1], torch.float32, dev)
    if dloss is not None:
        _same("dloss", dloss, h.shape[:-1], torch.float32, dev)
    dh = torch.empty_like(h) if want_dh else None
    dw = torch.empty_like(w) if want_dw else None
    nbytes = _workspace_bytes(qk_linear_xent_bwd_workspace_size, dev, M, V, K, code)
    ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=h.device)
    _check(load_library().qk_linear_xent_bwd(
        h.data_ptr(), w.data_ptr(), targets.data_ptr(), lse.data_ptr(), None if dloss is None else dloss.data_ptr(),
        dh.data_ptr() if want_dh else None, dw.data_ptr() if want_dw else None, ws.data_ptr(), nbytes, M, V, K, code,
        _options(ignore_index, z_loss), _current_stream(dev)), "qk_linear_xent_bwd")
    return dh, dw
