"""ctypes binding of libqk.so with the same names as the C ABI (include/qk.h).

Argument marshalling only: pointers, sizes, dtype codes and streams are
converted and passed through; the operators themselves run in the CUDA
kernels of libqk.so.  A non-OK status raises QkError.  There is no fallback:
if the library is missing every call raises.

The ``softmax_fwd`` / ``rmsnorm_fwd`` / ``layernorm_fwd`` / ``xent_fwd`` helpers take
and return CUDA tensors (they allocate the outputs with PyTorch and then call
the C entry points), and so do ``add_rmsnorm_fwd`` / ``add_rmsnorm_bwd`` /
``rmsnorm_quant_fwd`` / ``linear_xent_fwd`` / ``linear_xent_bwd`` / ``quant_fwd`` /
``scaled_mm_fwd`` / ``expert_sort`` / ``expert_gather_fwd`` / ``expert_combine_fwd`` /
``expert_combine_bwd``, which allocate their workspaces too.  A helper runs on
torch's current stream, or on the ``stream`` it is given, which has to have
waited for the inputs.
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
    "qk_linear_xent_bwd_workspace_size", "qk_quant_fwd", "qk_scaled_mm_fwd",
    "qk_scaled_mm_workspace_size", "qk_scaled_mm_get_plan", "qk_expert_sort", "qk_expert_sort_workspace_size",
    "qk_expert_gather_fwd", "qk_expert_combine_fwd", "qk_expert_combine_bwd",
)


class QkError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {qk_status_string(status)} (status {status})")


class qk_xent_options(ctypes.Structure):
    _fields_ = [("has_ignore_index", ctypes.c_int32), ("z_loss", ctypes.c_float),
                ("ignore_index", ctypes.c_int64)]


class qk_scaled_mm_plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "columns", "ctas", "grid")]


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
        sz = ctypes.c_size_t
        lib.qk_quant_fwd.argtypes = [vp] * 5 + [i64, i64, i64, i32, i32, vp]
        lib.qk_scaled_mm_workspace_size.argtypes = [i64, i64, i64, i64, sp]
        lib.qk_scaled_mm_get_plan.argtypes = [vp] * 2 + [i64] * 5 + [i32, ctypes.POINTER(qk_scaled_mm_plan)]
        lib.qk_scaled_mm_fwd.argtypes = [vp] * 7 + [sz, i64, i64, i64, i64, i64, i32, vp]
        lib.qk_expert_sort_workspace_size.argtypes = [i64, i64, i64, sp]
        lib.qk_expert_sort.argtypes = [vp, i64, vp, vp, vp, sz, i64, i64, i64, vp]
        lib.qk_expert_gather_fwd.argtypes = [vp] * 5 + [i64] * 5 + [vp]
        lib.qk_expert_combine_fwd.argtypes = [vp] * 4 + [i64] * 4 + [i32, vp]
        lib.qk_expert_combine_bwd.argtypes = [vp] * 6 + [i64] * 4 + [i32, vp]
        for name in ("qk_softmax_fwd", "qk_rmsnorm_fwd", "qk_xent_fwd", "qk_get_device_status",
                     "qk_get_plan", "qk_set_plan_override", "qk_test_wait_timeout",
                     "qk_softmax_bwd", "qk_rmsnorm_bwd_workspace_size", "qk_rmsnorm_bwd",
                     "qk_xent_bwd", "qk_rmsnorm_bwd_noalloc", "qk_xent_fwd_ex", "qk_xent_bwd_ex",
                     "qk_layernorm_fwd", "qk_add_rmsnorm_fwd", "qk_add_rmsnorm_bwd_workspace_size",
                     "qk_add_rmsnorm_bwd", "qk_rmsnorm_quant_fwd", "qk_linear_xent_fwd_workspace_size",
                     "qk_linear_xent_fwd", "qk_linear_xent_bwd_workspace_size", "qk_linear_xent_bwd",
                     "qk_quant_fwd", "qk_scaled_mm_workspace_size", "qk_scaled_mm_get_plan", "qk_scaled_mm_fwd",
                     "qk_expert_sort_workspace_size", "qk_expert_sort", "qk_expert_gather_fwd",
                     "qk_expert_combine_fwd", "qk_expert_combine_bwd"):
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


def qk_quant_fwd(x, q, scale, qt, scale_t, M: int, N: int, block_rows: int, dtype: int, qtype: int,
                 stream=None) -> None:
    _check(load_library().qk_quant_fwd(_ptr(x), _ptr(q), _ptr(scale), _ptr(qt), _ptr(scale_t), M, N, block_rows,
                                       dtype, qtype, _stream(stream)), "qk_quant_fwd")


def qk_scaled_mm_workspace_size(M: int, N: int, K: int, experts: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().qk_scaled_mm_workspace_size(M, N, K, experts, ctypes.byref(n)),
           "qk_scaled_mm_workspace_size")
    return n.value


def qk_scaled_mm_fwd(a, a_scale, b, b_scale, offsets, y, workspace, workspace_bytes: int, M: int, N: int, K: int,
                     experts: int, b_block_rows: int, out_dtype: int, stream=None) -> None:
    _check(load_library().qk_scaled_mm_fwd(_ptr(a), _ptr(a_scale), _ptr(b), _ptr(b_scale), _ptr(offsets), _ptr(y),
                                           _ptr(workspace), int(workspace_bytes), M, N, K, experts, b_block_rows,
                                           out_dtype, _stream(stream)), "qk_scaled_mm_fwd")


def qk_scaled_mm_get_plan(offsets, y, M: int, N: int, K: int, experts: int, b_block_rows: int,
                          out_dtype: int) -> dict:
    p = qk_scaled_mm_plan()
    _check(load_library().qk_scaled_mm_get_plan(_ptr(offsets), _ptr(y), M, N, K, experts, b_block_rows, out_dtype,
                                                ctypes.byref(p)), "qk_scaled_mm_get_plan")
    return {n: getattr(p, n) for n, _ in qk_scaled_mm_plan._fields_}


def qk_expert_sort_workspace_size(T: int, k: int, num_experts: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().qk_expert_sort_workspace_size(T, k, num_experts, ctypes.byref(n)),
           "qk_expert_sort_workspace_size")
    return n.value


def qk_expert_sort(experts, id_bytes: int, offsets, slot, workspace, workspace_bytes: int, T: int, k: int,
                   num_experts: int, stream=None) -> None:
    _check(load_library().qk_expert_sort(_ptr(experts), id_bytes, _ptr(offsets), _ptr(slot), _ptr(workspace),
                                         int(workspace_bytes), T, k, num_experts, _stream(stream)), "qk_expert_sort")


def qk_expert_gather_fwd(x, scale, slot, rows, row_scale, T: int, k: int, P: int, row_bytes: int, groups: int,
                         stream=None) -> None:
    _check(load_library().qk_expert_gather_fwd(_ptr(x), _ptr(scale), _ptr(slot), _ptr(rows), _ptr(row_scale), T, k,
                                               P, row_bytes, groups, _stream(stream)), "qk_expert_gather_fwd")


def qk_expert_combine_fwd(rows, slot, weights, y, T: int, k: int, P: int, N: int, dtype: int, stream=None) -> None:
    _check(load_library().qk_expert_combine_fwd(_ptr(rows), _ptr(slot), _ptr(weights), _ptr(y), T, k, P, N, dtype,
                                                _stream(stream)), "qk_expert_combine_fwd")


def qk_expert_combine_bwd(dy, rows, slot, weights, drows, dweights, T: int, k: int, P: int, N: int, dtype: int,
                          stream=None) -> None:
    _check(load_library().qk_expert_combine_bwd(_ptr(dy), _ptr(rows), _ptr(slot), _ptr(weights), _ptr(drows),
                                                _ptr(dweights), T, k, P, N, dtype, _stream(stream)),
           "qk_expert_combine_bwd")


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


def _device(x):
    """The device index of a CUDA tensor on the current device, as _matrix finds it."""
    global torch
    if torch is None:
        import torch as _torch
        torch = _torch
    dev = x.get_device()
    if dev < 0:
        raise ValueError("expected a CUDA tensor")
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"the tensors are on cuda:{dev}, the current device is cuda:{torch.cuda.current_device()}")
    return dev


def _blocks(n):
    return -(-n // 128)


def quant_fwd(x, block_rows: int = 1, qdtype=None, want_q: bool = True, want_t: bool = False, stream=None):
    """x [..., N] in 8 bits with a scale for each 128 columns of a row
    (block_rows 1) or each block of 128 x 128 (block_rows 128, x of two
    dimensions); returns (q, scale, qt, scale_t).  qt, with want_t, is x
    transposed in 8 bits (x of two dimensions), its scales along x's columns.
    Blocks count from x's first row: matrices stacked to one (experts' weights)
    have blocks of their own where each one's rows are a multiple of 128.
    What is not wanted is None.  qdtype as in rmsnorm_quant_fwd."""
    if stream is not None:
        return _on(stream, quant_fwd, x, block_rows, qdtype, want_q, want_t)
    M, N, code, dev = _matrix(x)
    if qdtype is None or qdtype is torch.float8_e4m3fn:
        qdtype, qcode = torch.float8_e4m3fn, QK_E4M3
    elif qdtype is torch.int8:
        qcode = QK_INT8
    else:
        raise TypeError(f"unsupported qdtype {qdtype}: torch.float8_e4m3fn or torch.int8 expected")
    if block_rows not in (1, 128):
        raise ValueError("block_rows must be 1 or 128")
    if not want_q and not want_t:
        raise ValueError("nothing is wanted")
    if (want_t or block_rows == 128) and x.dim() != 2:
        raise ValueError("blocks of rows and transposes need an x of two dimensions")
    shape, device = x.shape, x.device
    q = scale = qt = scale_t = None
    f32 = torch.float32
    if want_q:
        q = torch.empty(shape, dtype=qdtype, device=device)
        lead = shape[:-1] if block_rows == 1 else (_blocks(M),)
        scale = torch.empty(lead + (_blocks(N),), dtype=f32, device=device)
    if want_t:
        qt = torch.empty((N, M), dtype=qdtype, device=device)
        scale_t = torch.empty((N if block_rows == 1 else _blocks(N), _blocks(M)), dtype=f32, device=device)
    _check(load_library().qk_quant_fwd(
        x.data_ptr(), q.data_ptr() if want_q else None, scale.data_ptr() if want_q else None,
        qt.data_ptr() if want_t else None, scale_t.data_ptr() if want_t else None, M, N, block_rows, code, qcode,
        _current_stream(dev)), "qk_quant_fwd")
    return q, scale, qt, scale_t


def _scaled_mm_check(a, a_scale, b, b_scale, offsets, K, N, G, rows, experts, dev):
    e4m3, f32 = torch.float8_e4m3fn, torch.float32
    if a.dim() < 1 or b.dim() != (2 if offsets is None else 3):
        raise ValueError("b must be [N, K], or [experts, N, K] with offsets")
    if offsets is not None and a.dim() != 2:
        raise ValueError("a must be [rows, K] with offsets")
    _same("a", a, a.shape, e4m3, dev)
    _same("b", b, b.shape[:-1] + (K,), e4m3, dev)
    _same("a_scale", a_scale, a.shape[:-1] + (G,), f32, dev)
    if rows != N and rows != _blocks(N):
        raise ValueError(f"b_scale must have {_blocks(N)} or {N} rows")
    _same("b_scale", b_scale, b.shape[:-2] + (rows, G), f32, dev)
    if offsets is not None:
        _same("offsets", offsets, (experts + 1,), torch.int32, dev)


def scaled_mm_fwd(a, a_scale, b, b_scale, offsets=None, out_dtype=None, out=None, stream=None):
    """The product a @ b.T of 8-bit values (torch.float8_e4m3fn) with a scale for
    each block of 128 of the last axis: a [..., K] with a_scale [..., blocks], b
    [N, K] with b_scale [blocks of N, blocks] or [N, blocks].  With offsets
    (int32, from expert_sort) a is [rows, K], b [experts, N, K], and rows
    offsets[e] ... offsets[e + 1] - 1 are multiplied with b[e].T; rows behind
    the last are left as they were in `out`, and not written in a new tensor.
    The output is out_dtype, or out's (torch.bfloat16 or torch.float32; bfloat16
    when neither is given).  Operands that start off 16 bytes, or whose K is no
    multiple of 16, are copied on the way."""
    if stream is not None:
        return _on(stream, scaled_mm_fwd, a, a_scale, b, b_scale, offsets, out_dtype, out)
    dev = _device(a)
    shape = a.shape
    K, N = shape[-1] if shape else 0, b.shape[-2] if b.dim() > 1 else 0
    M, G = a.numel() // max(K, 1), -(-K // 128)
    rows = b_scale.shape[-2] if b_scale.dim() > 1 else -1
    experts = 1 if offsets is None else b.shape[0]
    # What most calls are, in a few comparisons; the full checks name what is wrong with others.
    e4m3, f32 = torch.float8_e4m3fn, torch.float32
    if not (a.dtype is e4m3 and b.dtype is e4m3 and a_scale.dtype is f32 and b_scale.dtype is f32 and K
            and shape == (M, K) and b.shape == (N, K) and a_scale.shape == (M, G) and b_scale.shape == (rows, G)
            and (rows == -(-N // 128) or rows == N) and offsets is None and a.is_contiguous() and b.is_contiguous()
            and a_scale.is_contiguous() and b_scale.is_contiguous() and b.get_device() == dev
            and a_scale.get_device() == dev and b_scale.get_device() == dev):
        _scaled_mm_check(a, a_scale, b, b_scale, offsets, K, N, G, rows, experts, dev)
    if out_dtype is None:
        out_dtype = torch.bfloat16 if out is None else out.dtype
    if out_dtype is torch.bfloat16:
        code = QK_BF16
    elif out_dtype is f32:
        code = QK_F32
    else:
        raise TypeError(f"unsupported out_dtype {out_dtype}: float32 or bfloat16 expected")
    y_shape = (M, N) if len(shape) == 2 else shape[:-1] + (N,)
    y = torch.empty(y_shape, dtype=out_dtype, device=a.device) if out is None else _same("out", out, y_shape,
                                                                                        out_dtype, dev)
    pa, pb, nbytes = a.data_ptr(), b.data_ptr(), 0
    if K % 16:
        nbytes = _workspace_bytes(qk_scaled_mm_workspace_size, dev, M, N, K, experts)
    elif (pa | pb) & 15:  # what starts off 16 bytes is copied
        nbytes = (a.numel() if pa & 15 else 0) + (b.numel() if pb & 15 else 0)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=a.device) if nbytes else None
    _check(load_library().qk_scaled_mm_fwd(
        pa, a_scale.data_ptr(), pb, b_scale.data_ptr(),
        None if offsets is None else offsets.data_ptr(), y.data_ptr(), ws.data_ptr() if nbytes else None, nbytes, M, N,
        K, experts, 1 if rows == N else 128, code, _current_stream(dev)), "qk_scaled_mm_fwd")
    return y


def expert_sort(experts, num_experts: int, stream=None):
    """Sorts the choices experts [T, k] (int32 or int64; outside [0, num_experts):
    none) by expert, in their order; returns (offsets, slot): int32 [num_experts + 1],
    where each expert's rows begin, and int32 [T, k], each choice's row (-1: none)."""
    if stream is not None:
        return _on(stream, expert_sort, experts, num_experts)
    dev = _device(experts)
    if experts.dim() != 2 or not experts.is_contiguous() or experts.dtype not in (torch.int32, torch.int64):
        raise ValueError("experts must be a contiguous int32 or int64 tensor [T, k]")
    if num_experts < 1:
        raise ValueError("num_experts must be positive")
    T, k = experts.shape
    offsets = torch.empty(num_experts + 1, dtype=torch.int32, device=experts.device)
    slot = torch.empty((T, k), dtype=torch.int32, device=experts.device)
    nbytes = _workspace_bytes(qk_expert_sort_workspace_size, dev, T, k, num_experts)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=experts.device) if nbytes else None
    _check(load_library().qk_expert_sort(
        experts.data_ptr(), 4 if experts.dtype is torch.int32 else 8, offsets.data_ptr(), slot.data_ptr(),
        ws.data_ptr() if nbytes else None, nbytes, T, k, num_experts, _current_stream(dev)), "qk_expert_sort")
    return offsets, slot


def _choices(slot, T, dev):
    shape = slot.shape
    if len(shape) != 2 or shape[0] != T:
        raise ValueError(f"slot must be [{T}, k]")
    if slot.dtype is not torch.int32 or not slot.is_contiguous() or slot.get_device() != dev:
        _same("slot", slot, shape, torch.int32, dev)
    return shape[1]


def expert_gather_fwd(x, slot, scale=None, out=None, out_scale=None, stream=None):
    """Copies each token's row x[t] to row slot[t, j] for each of its choices;
    returns the rows [T * k, N] (or out, [any number, N]).  With scale [T, groups]
    (float32, 8-bit rows) the scales move too, and (rows, row scales) is returned.
    Rows that no slot names are left as they were in `out`, and not written in a
    new tensor.  The gradient for x is expert_combine_fwd(drows, slot)."""
    if stream is not None:
        return _on(stream, expert_gather_fwd, x, slot, scale, out, out_scale)
    dev = _device(x)
    if x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous tensor [T, N]")
    T, N = x.shape
    k = _choices(slot, T, dev)
    rows = torch.empty((T * k, N), dtype=x.dtype, device=x.device) if out is None else out
    P = rows.shape[0]
    if out is not None:
        _same("out", out, (P, N), x.dtype, dev)
    groups, row_scale = 0, None
    if scale is not None:
        if scale.dim() != 2:
            raise ValueError("scale must be [T, groups]")
        groups = scale.shape[1]
        _same("scale", scale, (T, groups), torch.float32, dev)
        row_scale = (torch.empty((P, groups), dtype=torch.float32, device=x.device) if out_scale is None
                     else _same("out_scale", out_scale, (P, groups), torch.float32, dev))
    elif out_scale is not None:
        raise ValueError("out_scale needs a scale")
    _check(load_library().qk_expert_gather_fwd(
        x.data_ptr(), None if scale is None else scale.data_ptr(), slot.data_ptr(), rows.data_ptr(),
        None if scale is None else row_scale.data_ptr(), T, k, P, N * x.element_size(), groups, _current_stream(dev)),
        "qk_expert_gather_fwd")
    return rows if scale is None else (rows, row_scale)


def expert_combine_fwd(rows, slot, weights=None, out=None, stream=None):
    """Each token's sum over its choices of weights[t, j] * rows[slot[t, j]] (weights
    float32 [T, k], None: 1); choices without a slot are left out."""
    if stream is not None:
        return _on(stream, expert_combine_fwd, rows, slot, weights, out)
    P, N, code, dev = _matrix(rows)
    if rows.dim() != 2:
        raise ValueError("rows must be [rows, N]")
    T = slot.shape[0] if slot.dim() > 0 else 0
    k = _choices(slot, T, dev)
    if weights is not None:
        _same("weights", weights, (T, k), torch.float32, dev)
    y = torch.empty((T, N), dtype=rows.dtype, device=rows.device) if out is None else _same("out", out, (T, N),
                                                                                           rows.dtype, dev)
    _check(load_library().qk_expert_combine_fwd(
        rows.data_ptr(), slot.data_ptr(), None if weights is None else weights.data_ptr(), y.data_ptr(), T, k, P, N,
        code, _current_stream(dev)), "qk_expert_combine_fwd")
    return y


def expert_combine_bwd(dy, rows, slot, weights, out=None, want_dweights: bool = True, stream=None):
    """Backward of expert_combine_fwd; returns (drows, dweights) (dweights is None
    if not wanted).  out may be rows; rows that no slot names are left as they
    were in it, and not written in a new tensor."""
    if stream is not None:
        return _on(stream, expert_combine_bwd, dy, rows, slot, weights, out, want_dweights)
    T, N, code, dev = _matrix(dy)
    if dy.dim() != 2 or rows.dim() != 2:
        raise ValueError("dy must be [T, N] and rows [rows, N]")
    P = rows.shape[0]
    _same("rows", rows, (P, N), dy.dtype, dev)
    k = _choices(slot, T, dev)
    _same("weights", weights, (T, k), torch.float32, dev)
    drows = torch.empty_like(rows) if out is None else _same("out", out, (P, N), dy.dtype, dev)
    dweights = torch.empty((T, k), dtype=torch.float32, device=dy.device) if want_dweights else None
    _check(load_library().qk_expert_combine_bwd(
        dy.data_ptr(), rows.data_ptr(), slot.data_ptr(), weights.data_ptr(), drows.data_ptr(),
        dweights.data_ptr() if want_dweights else None, T, k, P, N, code, _current_stream(dev)),
        "qk_expert_combine_bwd")
    return drows, dweights
