"""Python binding of libzero_gb300.so, the ZeRO step on one GB300.

Argument marshalling only: every function below calls the C entry point of
the same name (declared in ``include/zero_step.h``) and turns a negative
status into :class:`ZeroError`.  Tensors may be passed wherever the C call
takes a device pointer (their ``data_ptr()`` is used) and torch streams
wherever it takes a ``cudaStream_t``.  All arithmetic runs in the library's
CUDA kernels; there is no fallback: if the library has not been built,
every call raises :class:`ZeroLibraryMissing`.

:class:`ZeroStep` is a convenience owner: it allocates the buffers a
configuration needs with PyTorch (the library itself allocates nothing),
places theta0 in the padded layout and creates the context.
"""

from __future__ import annotations

import array
import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libzero_gb300.so")

# constants of include/zero_step.h
ZERO_OK, ZERO_E_ARG, ZERO_E_ALIGN, ZERO_E_CUDA, ZERO_E_RANK, ZERO_E_TIMEOUT, ZERO_E_STATE = 0, -1, -2, -3, -4, -5, -6
ZERO_E_NOMEM = -7
ZERO_SCHEME_DP, ZERO_SCHEME_Z1, ZERO_SCHEME_Z2, ZERO_SCHEME_Z3 = 0, 1, 2, 3
ZERO_FP16, ZERO_BF16, ZERO_FP32 = 0, 1, 2
ZERO_RESIDENT, ZERO_PEAK = 0, 1
ZERO_VARIANT_AUTO, ZERO_VARIANT_VECTOR, ZERO_VARIANT_BULK = 0, 1, 2
(ZERO_STAT_COMM_BYTES, ZERO_STAT_LAUNCHES, ZERO_STAT_GATHERS, ZERO_STAT_SCATTERS, ZERO_STAT_LIVE_ELEMS,
 ZERO_STAT_PEAK_LIVE_ELEMS, ZERO_STAT_T, ZERO_STAT_DEVICE_ERRORS, ZERO_STAT_LAST_VARIANT) = range(9)
ZERO_MAX_RANKS = 64
ZERO_KERNEL_FUSED, ZERO_KERNEL_GATHER, ZERO_KERNEL_CAST, ZERO_KERNEL_NORM = 0, 1, 2, 3
ZERO_DEBUG_POISON_RELEASED = 1

# (a, b, c) of each Newton-Schulz step as Muon's authors published them: they take singular values from about 1e-2
# up to between 0.7 and 1.2 in five steps
MUON_COEFFICIENTS = ((3.4445, -4.7750, 2.0315),) * 5

ERROR_NAMES = {ZERO_E_ARG: "ZERO_E_ARG", ZERO_E_ALIGN: "ZERO_E_ALIGN", ZERO_E_CUDA: "ZERO_E_CUDA",
               ZERO_E_RANK: "ZERO_E_RANK", ZERO_E_TIMEOUT: "ZERO_E_TIMEOUT", ZERO_E_STATE: "ZERO_E_STATE",
               ZERO_E_NOMEM: "ZERO_E_NOMEM"}

# every symbol the header declares, with (restype, argtypes)
_P, _I, _L, _D = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_double
_PP = ctypes.POINTER(ctypes.c_void_p)
_LP = ctypes.POINTER(ctypes.c_int64)
HOOK = ctypes.CFUNCTYPE(None, ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p)
SIGNATURES = {
    "zero_buffer_sizes": (_I, [_I, _I, _L, _LP, _LP]),
    "zero_layout": (_I, [_I, _L, _LP, _LP, _LP, _LP]),
    "zero_bytes_per_rank": (_L, [_I, _L, _I, _I, _L]),
    "zero_comm_bytes_closed_form": (_L, [_I, _L, _I]),
    "zero_init": (_I, [ctypes.POINTER(_P), _I, _I, _L, _L, _LP, _I, _I, _P, _P, _P, _P, _PP, _PP, _P, _P]),
    "zero_destroy": (_I, [_P]),
    "zero_refresh_working_copy": (_I, [_P]),
    "zero_step": (_I, [_P, _I, _I, _L, _PP, _D, _D, _D, _D, _L]),
    "zero_set_unit_hook": (_I, [_P, HOOK, _P]),
    "zero_step_bucket": (_I, [_P, _L, _L, _PP, _D, _D, _D, _D, _L, _P]),
    "zero_host_staging_bytes": (_L, [_I, _I, _L, _LP, _L]),
    "zero_step_host": (_I, [_P, _I, _I, _L, _PP, _P, _P, _L, _L, _D, _D, _D, _D, _L, _P, _P]),
    "zero_offload_staging_bytes": (_L, [_L]),
    "zero_offload_init": (_I, [ctypes.POINTER(_P), _I, _L, _I, _I, _P, _P, _P, _P, _P, _P, _P, _L, _L, _I, _P]),
    "zero_offload_step": (_I, [_P, _PP, _D, _D, _D, _D, _L]),
    "zero_offload_stats": (_I, [_P, _LP, ctypes.POINTER(ctypes.c_double), _LP, _LP, _LP,
                                ctypes.POINTER(ctypes.c_int)]),
    "zero_offload_destroy": (_I, [_P]),
    "zero_offload_set_step": (_I, [_P, _L]),
    "zero_adam_host": (_I, [_L, _P, _P, _P, _P, _P, _I, _D, _D, _D, _D, _L, _I, _I]),
    "zero_host_alloc": (_I, [_L, ctypes.POINTER(_P)]),
    "zero_host_free": (_I, [_P]),
    "zero_gather_unit": (_I, [_P, _L, _P, _P]),
    "zero_release_unit": (_I, [_P, _L]),
    "zero_update_unit": (_I, [_P, _L, _PP, _D, _D, _D, _D, _L, _P]),
    "zero_get_state": (_I, [_P, _P, _P, _P, _LP]),
    "zero_set_state": (_I, [_P, _P, _P, _P, _L]),
    "zero_comm_bytes_per_rank": (_L, [_P]),
    "zero_stat": (_L, [_P, _I]),
    "zero_sync": (_I, [_P, _I]),
    "zero_enable_timing": (_I, [_P, _I]),
    "zero_read_timing": (_I, [_P, _I, ctypes.POINTER(ctypes.c_double), _LP]),
    "zero_set_variant": (_I, [_P, _I]),
    "zero_set_graph": (_I, [_P, _I]),
    "zero_inject_stall": (_I, [_P, _L]),
    "zero_set_debug": (_I, [_P, _I]),
    "zero_mark_rank": (_I, [_P, _I, _I]),
    "zero_step_z3_static": (_I, [_I, _L, _LP, _I, _I, _P, _P, _P, _PP, _PP, _D, _D, _D, _D, _L, HOOK, _P, _P]),
    "zero_step_dp_replicas": (_I, [_I, _L, _I, _I, _PP, _PP, _PP, _PP, _PP, _D, _D, _D, _D, _L, _P]),
    "zero_dp_replicas_mismatches": (_I, [_I, _L, _PP, _PP, _PP, _PP, _P, _P]),
    "zero_grad_norm_workspace_bytes": (_L, []),
    "zero_grad_norm": (_I, [_I, _L, _P, _I, _P, _P, _P, _L, _P]),
    "zero_grad_clip": (_I, [_I, _L, _P, _I, _P, _P, _D, _P, _P]),
    "zero_step_clipped_workspace_bytes": (_L, [_P]),
    "zero_step_clipped": (_I, [_P, _I, _I, _L, _PP, _D, _D, _D, _D, _L, _D, _P, _P, _L]),
    "zero_embedding": (_I, [_L, _L, _L, _I, _P, _I, _P, _L, _D, _P, _L, _P]),
    "zero_embedding_workspace_bytes": (_L, [_L, _L]),
    "zero_embedding_grad": (_I, [_L, _L, _L, _I, _P, _I, _P, _L, _D, _P, _L, _I, _P, _L, _P]),
    "zero_lm_workspace_bytes": (_L, [_L, _L, _L, _I]),
    "zero_lm_loss": (_I, [_L, _L, _L, _I, _P, _L, _P, _L, _P, _I, _P, _P, _P, _L, _P]),
    "zero_lm_loss_grad": (_I, [_L, _L, _L, _I, _P, _L, _P, _L, _P, _I, _P, _D, _P, _L, _P, _L, _I, _P, _L, _P]),
    "zero_lm_logprobs_workspace_bytes": (_L, [_L, _L, _L, _I, _I]),
    "zero_lm_logprobs": (_I, [_L, _L, _L, _I, _P, _L, _P, _L, _P, _I, _D, _I, _P, _P, _P, _P, _P, _P, _L, _P]),
    "zero_lm_logprobs_grad": (_I, [_L, _L, _L, _I, _P, _L, _P, _L, _P, _I, _D, _P, _P, _P, _P, _P, _L, _P, _L, _I, _P,
                                   _L, _P]),
    "zero_orthogonalize_workspace_bytes": (_L, [_L, _P, _P]),
    "zero_orthogonalize": (_I, [_L, _P, _P, _I, _P, _P, _P, _P, _I, _P, _I, _P, _L, _P]),
    "zero_muon_workspace_bytes": (_L, [_I, _L, _P, _P]),
    "zero_muon_step": (_I, [_I, _L, _P, _P, _I, _I, _P, _P, _P, _P, _D, _D, _I, _D, _P, _I, _P, _I, _P, _L, _P]),
    "zero_lm_workspace_status": (_I, [_P, _P]),
    "zero_lm_status": (_I, [_P]),
    "zero_lm_inject_stall": (_I, []),
    "zero_last_error": (ctypes.c_char_p, []),
}


class ZeroLibraryMissing(ImportError):
    pass


class ZeroError(RuntimeError):
    def __init__(self, code: int, func: str, message: str):
        super().__init__(f"{func}: {ERROR_NAMES.get(code, code)}: {message}")
        self.code = code


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library (loaded on first use; raises if it is not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ZeroLibraryMissing(
                f"{LIB_PATH} is not built; build it with `python -m zero_sharded_mixed_step_gb300.build`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def _check(name: str, rc: int) -> int:
    if rc < 0:
        raise ZeroError(rc, name, lib().zero_last_error().decode())
    return rc


def _ptr(x):
    if x is None:
        return None
    if hasattr(x, "data_ptr"):
        # the library reads and writes dense vectors from this address
        if hasattr(x, "is_contiguous") and not x.is_contiguous():
            raise ValueError("a tensor passed to the library must be contiguous")
        return x.data_ptr()
    return int(x)


def _addr(x):
    """The address of a tensor whose rows the caller describes by a stride."""
    return x.data_ptr() if hasattr(x, "data_ptr") else x


def _stream(s):
    if s is None:
        return None
    if hasattr(s, "cuda_stream"):
        return s.cuda_stream or None
    return int(s) or None


def _ptr_array(xs):
    if xs is None:
        return None
    return (ctypes.c_void_p * len(xs))(*[_ptr(x) for x in xs])


def _i64_array(xs):
    return (ctypes.c_int64 * len(xs))(*[int(x) for x in xs])


# ---- the entry points, same names as the C ABI --------------------------------

def zero_last_error() -> str:
    return lib().zero_last_error().decode()


def zero_buffer_sizes(scheme: int, W: int, unit_sizes) -> dict:
    out = (ctypes.c_int64 * 6)()
    _check("zero_buffer_sizes", lib().zero_buffer_sizes(scheme, W, len(unit_sizes), _i64_array(unit_sizes), out))
    return dict(n=out[0], n_pad=out[1], p16=out[2], shard_store=out[3], unit_buf=out[4], units=out[5])


def zero_layout(W: int, unit_sizes):
    U = len(unit_sizes)
    off, shard, off16 = (ctypes.c_int64 * U)(), (ctypes.c_int64 * U)(), (ctypes.c_int64 * U)()
    _check("zero_layout", lib().zero_layout(W, U, _i64_array(unit_sizes), off, shard, off16))
    return list(off), list(shard), list(off16)


def zero_bytes_per_rank(scheme: int, n: int, W: int, kind: int = ZERO_RESIDENT, gathered_elems: int = 0) -> int:
    return _check("zero_bytes_per_rank", lib().zero_bytes_per_rank(scheme, n, W, kind, gathered_elems))


def zero_comm_bytes_closed_form(scheme: int, n: int, W: int) -> int:
    return _check("zero_comm_bytes_closed_form", lib().zero_comm_bytes_closed_form(scheme, n, W))


def zero_init(scheme, W, n, unit_sizes, grad_dtype, work_dtype, master, m, v, p16=None, shard16=None,
              unit_bufs=None, stream_update=None, stream_gather=None) -> int:
    ctx = ctypes.c_void_p()
    _check("zero_init", lib().zero_init(
        ctypes.byref(ctx), scheme, W, n, len(unit_sizes), _i64_array(unit_sizes), grad_dtype, work_dtype,
        _ptr(master), _ptr(m), _ptr(v), _ptr(p16), _ptr_array(shard16), _ptr_array(unit_bufs),
        _stream(stream_update), _stream(stream_gather)))
    return ctx.value


def zero_destroy(ctx) -> None:
    _check("zero_destroy", lib().zero_destroy(ctx))


def zero_refresh_working_copy(ctx) -> None:
    _check("zero_refresh_working_copy", lib().zero_refresh_working_copy(ctx))


def zero_step(ctx, scheme, W, n, grads, lr, beta1, beta2, eps, t) -> None:
    _check("zero_step", lib().zero_step(ctx, scheme, W, n, _ptr_array(grads), lr, beta1, beta2, eps, t))


def zero_step_bucket(ctx, lo, length, bucket_grads, lr, beta1, beta2, eps, t, stream=None) -> None:
    _check("zero_step_bucket", lib().zero_step_bucket(ctx, lo, length, _ptr_array(bucket_grads), lr, beta1, beta2, eps,
                                                      t, _stream(stream)))


def zero_host_staging_bytes(scheme, W, unit_sizes, chunk_elems=0) -> int:
    return _check("zero_host_staging_bytes", lib().zero_host_staging_bytes(
        scheme, W, len(unit_sizes), _i64_array(unit_sizes), chunk_elems))


def zero_step_host(ctx, scheme, W, n, host_grads, host_out, staging, staging_bytes, chunk_elems,
                   lr, beta1, beta2, eps, t, stream_h2d=None, stream_d2h=None) -> None:
    """host_grads: W host buffers (tensors or addresses); host_out: host buffer or None."""
    _check("zero_step_host", lib().zero_step_host(
        ctx, scheme, W, n, _ptr_array(host_grads), _ptr(host_out), _ptr(staging), staging_bytes, chunk_elems,
        lr, beta1, beta2, eps, t, _stream(stream_h2d), _stream(stream_d2h)))


def zero_host_alloc(nbytes: int) -> int:
    """Page-locked host memory on huge pages for the host-fed step; returns its address."""
    p = ctypes.c_void_p()
    _check("zero_host_alloc", lib().zero_host_alloc(int(nbytes), ctypes.byref(p)))
    return p.value


def zero_host_free(ptr) -> None:
    _check("zero_host_free", lib().zero_host_free(ptr))


def zero_offload_staging_bytes(chunk_elems: int = 0) -> int:
    return _check("zero_offload_staging_bytes", lib().zero_offload_staging_bytes(chunk_elems))


def zero_offload_init(W, n, grad_dtype, work_dtype, host_master, host_m, host_v, host_grad, host_p16, p16,
                      staging, staging_bytes, chunk_elems=0, threads=0, stream=None):
    ctx = ctypes.c_void_p()
    _check("zero_offload_init", lib().zero_offload_init(
        ctypes.byref(ctx), W, n, grad_dtype, work_dtype, _ptr(host_master), _ptr(host_m), _ptr(host_v),
        _ptr(host_grad), _ptr(host_p16), _ptr(p16), _ptr(staging), staging_bytes, chunk_elems, threads,
        _stream(stream)))
    return ctx


def zero_offload_step(ctx, grads, lr, beta1, beta2, eps, t) -> None:
    _check("zero_offload_step", lib().zero_offload_step(ctx, _ptr_array(grads), lr, beta1, beta2, eps, t))


def zero_offload_stats(ctx) -> dict:
    t, d2h, h2d, launches = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    secs, threads = ctypes.c_double(), ctypes.c_int()
    _check("zero_offload_stats", lib().zero_offload_stats(ctx, ctypes.byref(t), ctypes.byref(secs),
                                                          ctypes.byref(d2h), ctypes.byref(h2d),
                                                          ctypes.byref(launches), ctypes.byref(threads)))
    return {"t": t.value, "host_seconds": secs.value, "d2h_bytes": d2h.value, "h2d_bytes": h2d.value,
            "launches": launches.value, "threads": threads.value}


def zero_offload_set_step(ctx, t: int) -> None:
    _check("zero_offload_set_step", lib().zero_offload_set_step(ctx, t))


def zero_offload_destroy(ctx) -> None:
    _check("zero_offload_destroy", lib().zero_offload_destroy(ctx))


def zero_adam_host(n, grad, master, m, v, out16, work_dtype, lr, beta1, beta2, eps, t, W=1, threads=0) -> None:
    """The offloaded step's host update on host tensors (no GPU needed)."""
    _check("zero_adam_host", lib().zero_adam_host(n, _ptr(grad), _ptr(master), _ptr(m), _ptr(v), _ptr(out16),
                                                  work_dtype, lr, beta1, beta2, eps, t, W, threads))


class HostBuffer:
    """A zero_host_alloc block seen as a CPU tensor of ``numel`` values of
    ``dtype`` (the tensor shares the memory; keep this object alive while it
    or any copy in flight uses it, then ``close()``)."""

    def __init__(self, numel: int, dtype):
        import torch
        itemsize = torch.empty(0, dtype=dtype).element_size()
        self.nbytes = max(1, int(numel) * itemsize)
        self.ptr = zero_host_alloc(self.nbytes)
        raw = (ctypes.c_uint8 * self.nbytes).from_address(self.ptr)
        self.tensor = torch.frombuffer(raw, dtype=torch.uint8)[: int(numel) * itemsize].view(dtype)

    def close(self):
        if self.ptr:
            self.tensor = None
            zero_host_free(self.ptr)
            self.ptr = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def zero_set_unit_hook(ctx, fn, user=None):
    """``fn(user, phase, unit, unit_buf, stream)``; returns the ctypes callback,
    which the caller must keep alive while it is registered."""
    cb = HOOK(fn) if fn is not None else HOOK()
    _check("zero_set_unit_hook", lib().zero_set_unit_hook(ctx, cb, user))
    return cb


def zero_gather_unit(ctx, unit, dst, stream=None) -> None:
    _check("zero_gather_unit", lib().zero_gather_unit(ctx, unit, _ptr(dst), _stream(stream)))


def zero_release_unit(ctx, unit) -> None:
    _check("zero_release_unit", lib().zero_release_unit(ctx, unit))


def zero_update_unit(ctx, unit, grads, lr, beta1, beta2, eps, t, stream=None) -> None:
    _check("zero_update_unit", lib().zero_update_unit(ctx, unit, _ptr_array(grads), lr, beta1, beta2, eps, t,
                                                      _stream(stream)))


def zero_get_state(ctx, master=None, m=None, v=None) -> int:
    t = ctypes.c_int64()
    _check("zero_get_state", lib().zero_get_state(ctx, _ptr(master), _ptr(m), _ptr(v), ctypes.byref(t)))
    return t.value


def zero_set_state(ctx, master, m, v, t) -> None:
    _check("zero_set_state", lib().zero_set_state(ctx, _ptr(master), _ptr(m), _ptr(v), t))


def zero_comm_bytes_per_rank(ctx) -> int:
    return _check("zero_comm_bytes_per_rank", lib().zero_comm_bytes_per_rank(ctx))


def zero_stat(ctx, which: int) -> int:
    return _check("zero_stat", lib().zero_stat(ctx, which))


def zero_sync(ctx, timeout_ms: int = -1) -> None:
    _check("zero_sync", lib().zero_sync(ctx, timeout_ms))


def zero_enable_timing(ctx, on: bool) -> None:
    _check("zero_enable_timing", lib().zero_enable_timing(ctx, 1 if on else 0))


def zero_read_timing(ctx, kernel: int):
    """(total milliseconds, launches) of the timed launches of ``kernel`` since the last read."""
    ms, k = ctypes.c_double(), ctypes.c_int64()
    _check("zero_read_timing", lib().zero_read_timing(ctx, kernel, ctypes.byref(ms), ctypes.byref(k)))
    return ms.value, k.value


def zero_set_variant(ctx, variant: int) -> None:
    _check("zero_set_variant", lib().zero_set_variant(ctx, variant))


def zero_set_graph(ctx, on: bool) -> None:
    _check("zero_set_graph", lib().zero_set_graph(ctx, 1 if on else 0))


def zero_set_debug(ctx, flags: int) -> None:
    _check("zero_set_debug", lib().zero_set_debug(ctx, flags))


def zero_inject_stall(ctx, tile: int) -> None:
    _check("zero_inject_stall", lib().zero_inject_stall(ctx, tile))


def zero_mark_rank(ctx, rank: int, available: bool) -> None:
    _check("zero_mark_rank", lib().zero_mark_rank(ctx, rank, 1 if available else 0))


def zero_step_z3_static(W, unit_sizes, grad_dtype, work_dtype, master, m, v, shard16, grads,
                        lr, beta1, beta2, eps, t, hook=None, stream=None) -> None:
    """The ZeRO-3 step for callers that cannot allocate device memory: its
    gather buffer is the library's own fixed array (units up to 8,388,608
    padded 16-bit values); no context."""
    cb = HOOK(hook) if hook is not None else HOOK()
    _check("zero_step_z3_static", lib().zero_step_z3_static(
        W, len(unit_sizes), _i64_array(unit_sizes), grad_dtype, work_dtype, _ptr(master), _ptr(m), _ptr(v),
        _ptr_array(shard16), _ptr_array(grads), lr, beta1, beta2, eps, t, cb, None, _stream(stream)))


def zero_step_dp_replicas(W, n, grad_dtype, work_dtype, grads, master, m, v, p16, lr, beta1, beta2, eps, t,
                          stream=None) -> None:
    """One DP step over W literal replicas (lists of W device buffers each);
    no context, the caller keeps t."""
    _check("zero_step_dp_replicas", lib().zero_step_dp_replicas(
        W, n, grad_dtype, work_dtype, _ptr_array(grads), _ptr_array(master), _ptr_array(m), _ptr_array(v),
        _ptr_array(p16), lr, beta1, beta2, eps, t, _stream(stream)))


def zero_dp_replicas_mismatches(W, n, master, m, v, p16, mismatches, stream=None) -> None:
    """Enqueue the bitwise comparison of every replica with replica 0; the
    count lands in the device int64 ``mismatches``."""
    _check("zero_dp_replicas_mismatches", lib().zero_dp_replicas_mismatches(
        W, n, _ptr_array(master), _ptr_array(m), _ptr_array(v), _ptr_array(p16), _ptr(mismatches),
        _stream(stream)))


def _u64_array(values):
    """The values as a C array of 64-bit words and its address."""
    a = array.array("Q", values)
    return a, a.buffer_info()[0]


def zero_grad_norm_workspace_bytes() -> int:
    return lib().zero_grad_norm_workspace_bytes()


def zero_grad_norm(W, numels, dtype, grads, norm, workspace, workspace_bytes, stream=None) -> None:
    """grads: W * len(numels) device pointers or tensors, rank after rank."""
    sizes, sizes_at = _u64_array(numels)
    ptrs, ptrs_at = _u64_array([_ptr(g) or 0 for g in grads])
    _check("zero_grad_norm", lib().zero_grad_norm(W, len(sizes), sizes_at, dtype, ptrs_at, _ptr(norm),
                                                  _ptr(workspace), workspace_bytes, _stream(stream)))


def zero_grad_clip(W, numels, dtype, grads, norm, max_norm, out, stream=None) -> None:
    sizes, sizes_at = _u64_array(numels)
    ptrs, ptrs_at = _u64_array([_ptr(g) or 0 for g in grads])
    outs, outs_at = _u64_array([_ptr(o) or 0 for o in out])
    _check("zero_grad_clip", lib().zero_grad_clip(W, len(sizes), sizes_at, dtype, ptrs_at, _ptr(norm), max_norm,
                                                  outs_at, _stream(stream)))


def zero_step_clipped_workspace_bytes(ctx) -> int:
    return _check("zero_step_clipped_workspace_bytes", lib().zero_step_clipped_workspace_bytes(ctx))


def zero_step_clipped(ctx, scheme, W, n, grads, lr, beta1, beta2, eps, t, max_norm, norm, workspace,
                      workspace_bytes) -> None:
    _check("zero_step_clipped", lib().zero_step_clipped(ctx, scheme, W, n, _ptr_array(grads), lr, beta1, beta2, eps, t,
                                                        max_norm, _ptr(norm), _ptr(workspace), workspace_bytes))


def zero_embedding(tokens, vocab, width, dtype, ids, id_bytes, table, table_stride, scale, out, out_stride,
                   stream=None) -> None:
    _check("zero_embedding", lib().zero_embedding(tokens, vocab, width, dtype, _addr(ids), id_bytes, _addr(table),
                                                  table_stride, scale, _addr(out), out_stride, _stream(stream)))


def zero_embedding_workspace_bytes(tokens: int, width: int) -> int:
    return _check("zero_embedding_workspace_bytes", lib().zero_embedding_workspace_bytes(tokens, width))


def zero_embedding_grad(tokens, vocab, width, dtype, ids, id_bytes, dout, dout_stride, scale, dtable, dtable_stride,
                        accumulate, workspace, workspace_bytes, stream=None) -> None:
    _check("zero_embedding_grad", lib().zero_embedding_grad(
        tokens, vocab, width, dtype, _addr(ids), id_bytes, _addr(dout), dout_stride, scale, _addr(dtable),
        dtable_stride, 1 if accumulate else 0, _addr(workspace), workspace_bytes, _stream(stream)))


def zero_lm_workspace_bytes(tokens: int, vocab: int, width: int, with_grad: bool = True) -> int:
    return _check("zero_lm_workspace_bytes", lib().zero_lm_workspace_bytes(tokens, vocab, width, 1 if with_grad else 0))


def zero_lm_loss(tokens, vocab, width, dtype, hidden, hidden_stride, table, table_stride, targets, id_bytes, loss, lse,
                 workspace, workspace_bytes, stream=None) -> None:
    _check("zero_lm_loss", lib().zero_lm_loss(
        tokens, vocab, width, dtype, _addr(hidden), hidden_stride, _addr(table), table_stride, _addr(targets),
        id_bytes, _addr(loss), _addr(lse), _addr(workspace), workspace_bytes, _stream(stream)))


def zero_lm_loss_grad(tokens, vocab, width, dtype, hidden, hidden_stride, table, table_stride, targets, id_bytes, lse,
                      scale, dhidden, dhidden_stride, dtable, dtable_stride, accumulate, workspace, workspace_bytes,
                      stream=None) -> None:
    _check("zero_lm_loss_grad", lib().zero_lm_loss_grad(
        tokens, vocab, width, dtype, _addr(hidden), hidden_stride, _addr(table), table_stride, _addr(targets),
        id_bytes, _addr(lse), scale, _addr(dhidden), dhidden_stride, _addr(dtable), dtable_stride,
        1 if accumulate else 0, _addr(workspace), workspace_bytes, _stream(stream)))


def zero_lm_logprobs_workspace_bytes(tokens: int, vocab: int, width: int, top: int = 0, with_grad: bool = True) -> int:
    return _check("zero_lm_logprobs_workspace_bytes", lib().zero_lm_logprobs_workspace_bytes(
        tokens, vocab, width, top, 1 if with_grad else 0))


def zero_lm_logprobs(tokens, vocab, width, dtype, hidden, hidden_stride, table, table_stride, targets, id_bytes, scale,
                     top, logp, entropy, lse, top_logp, top_ids, workspace, workspace_bytes, stream=None) -> None:
    _check("zero_lm_logprobs", lib().zero_lm_logprobs(
        tokens, vocab, width, dtype, _addr(hidden), hidden_stride, _addr(table), table_stride, _addr(targets), id_bytes,
        scale, top, _addr(logp), _addr(entropy), _addr(lse), _addr(top_logp), _addr(top_ids), _addr(workspace),
        workspace_bytes, _stream(stream)))


def zero_lm_logprobs_grad(tokens, vocab, width, dtype, hidden, hidden_stride, table, table_stride, targets, id_bytes,
                          scale, lse, dlogp, entropy, dentropy, dhidden, dhidden_stride, dtable, dtable_stride,
                          accumulate, workspace, workspace_bytes, stream=None) -> None:
    _check("zero_lm_logprobs_grad", lib().zero_lm_logprobs_grad(
        tokens, vocab, width, dtype, _addr(hidden), hidden_stride, _addr(table), table_stride, _addr(targets), id_bytes,
        scale, _addr(lse), _addr(dlogp), _addr(entropy), _addr(dentropy), _addr(dhidden), dhidden_stride, _addr(dtable),
        dtable_stride, accumulate, _addr(workspace), workspace_bytes, _stream(stream)))


def _c_array(code, values):
    """The values as a C array of the given type code and its address."""
    a = array.array(code, values)
    return a, a.buffer_info()[0]


def _shape_arrays(shapes):
    rows, rows_at = _c_array("q", [r for r, _ in shapes])
    cols, cols_at = _c_array("q", [c for _, c in shapes])
    return (rows, cols), rows_at, cols_at


def _steps_of(coefficients):
    """(number of steps, array, address) of rows (a, b, c)."""
    rows = [tuple(map(float, row)) for row in coefficients]
    if any(len(row) != 3 for row in rows):
        raise ValueError("coefficients must be rows (a, b, c), one for each step")
    a, at = _c_array("d", [x for row in rows for x in row])
    return len(rows), a, at


def zero_orthogonalize_workspace_bytes(shapes) -> int:
    keep, rows, cols = _shape_arrays(shapes)
    return _check("zero_orthogonalize_workspace_bytes", lib().zero_orthogonalize_workspace_bytes(len(shapes), rows, cols))


def zero_orthogonalize(shapes, dtype, matrices, in_strides, out, out_strides, coefficients, fine_steps, workspace,
                       workspace_bytes, stream=None) -> None:
    """``in_strides`` and ``out_strides`` may be None (contiguous rows)."""
    keep, rows, cols = _shape_arrays(shapes)
    ins, ins_at = _u64_array([_addr(x) or 0 for x in matrices])
    outs, outs_at = _u64_array([_addr(x) or 0 for x in out])
    si, si_at = (None, None) if in_strides is None else _c_array("q", in_strides)
    so, so_at = (None, None) if out_strides is None else _c_array("q", out_strides)
    steps, co, co_at = _steps_of(coefficients)
    _check("zero_orthogonalize", lib().zero_orthogonalize(
        len(shapes), rows, cols, dtype, ins_at, si_at, outs_at, so_at, steps, co_at, fine_steps, _addr(workspace),
        workspace_bytes, _stream(stream)))


def zero_muon_workspace_bytes(W, shapes) -> int:
    keep, rows, cols = _shape_arrays(shapes)
    return _check("zero_muon_workspace_bytes", lib().zero_muon_workspace_bytes(W, len(shapes), rows, cols))


def zero_muon_step(W, shapes, grad_dtype, work_dtype, grads, master, momentum, p16, lr, mu, nesterov, weight_decay,
                   scales, coefficients, fine_steps, workspace, workspace_bytes, stream=None) -> None:
    """``grads``: W lists of matrices; ``scales`` may be None (1 for every matrix)."""
    keep, rows, cols = _shape_arrays(shapes)
    lists = [_u64_array([_addr(x) or 0 for x in xs]) for xs in ([g for rank in grads for g in rank], master, momentum, p16)]
    sc, sc_at = (None, None) if scales is None else _c_array("d", scales)
    steps, co, co_at = _steps_of(coefficients)
    _check("zero_muon_step", lib().zero_muon_step(
        W, len(shapes), rows, cols, grad_dtype, work_dtype, *(at for _, at in lists), lr, mu, 1 if nesterov else 0,
        weight_decay, sc_at, steps, co_at, fine_steps, _addr(workspace), workspace_bytes, _stream(stream)))


def zero_lm_workspace_status(workspace, stream=None) -> None:
    """Wait for the stream; raises ZeroError if a bounded device wait of a call with this workspace gave up."""
    _check("zero_lm_workspace_status", lib().zero_lm_workspace_status(_addr(workspace), _stream(stream)))


def zero_lm_status(stream=None) -> None:
    """Wait for the stream; raises ZeroError if a bounded device wait of any LM call on the device gave up."""
    _check("zero_lm_status", lib().zero_lm_status(_stream(stream)))


def zero_lm_inject_stall() -> None:
    """Testing: this thread's next LM call loses a block of operands, and its waits run out."""
    _check("zero_lm_inject_stall", lib().zero_lm_inject_stall())


# ---- convenience owners ---------------------------------------------------------

_DT = {"fp16": ZERO_FP16, "bf16": ZERO_BF16, ZERO_FP16: ZERO_FP16, ZERO_BF16: ZERO_BF16}


def _zeros_on(device):
    """The owners' allocator; it holds no owner, whose buffers are then freed with it and not by the next collection."""
    import torch
    return lambda numel, dtype: torch.zeros(numel, dtype=dtype, device=device)


class ZeroStep:
    """Buffers for one configuration, allocated with PyTorch on ``device``,
    plus the library context that uses them.

    ``theta0`` (n fp32 values, any device) is written to the real positions
    of the padded master; m and v start at zero; the 16-bit working copy is
    cast from the master before the first step.  ``alloc(numel, dtype)``, if
    given, supplies every device buffer instead of ``torch.zeros`` (a
    zero-filled tensor on ``device``, e.g. from the caller's own pool).
    """

    def __init__(self, scheme, W, unit_sizes, grad_dtype="fp16", work_dtype=None, theta0=None,
                 device="cuda", stream=None, gather_stream=None, with_grad_buffers=False, alloc=None):
        import torch
        self.torch = torch
        self.scheme, self.W = int(scheme), int(W)
        self.unit_sizes = [int(s) for s in unit_sizes]
        self.gdt = _DT[grad_dtype]
        self.wdt = _DT[work_dtype if work_dtype is not None else grad_dtype]
        self.sizes = zero_buffer_sizes(self.scheme, self.W, self.unit_sizes)
        self.n, self.n_pad = self.sizes["n"], self.sizes["n_pad"]
        self.off, self.shard, self.off16 = zero_layout(self.W, self.unit_sizes)
        self.device = torch.device(device)
        t16 = {ZERO_FP16: torch.float16, ZERO_BF16: torch.bfloat16}
        self.grad_torch_dtype, self.work_torch_dtype = t16[self.gdt], t16[self.wdt]
        self._alloc = alloc or _zeros_on(self.device)
        f32, w16 = torch.float32, self.work_torch_dtype
        self.master = self._alloc(self.n_pad, f32)
        self.m = self._alloc(self.n_pad, f32)
        self.v = self._alloc(self.n_pad, f32)
        self.p16 = self._alloc(self.sizes["p16"], w16) if self.scheme != ZERO_SCHEME_Z3 else None
        self.shard16 = ([self._alloc(self.sizes["shard_store"], w16) for _ in range(self.W)]
                        if self.scheme == ZERO_SCHEME_Z3 else None)
        self.unit_bufs = ([self._alloc(self.sizes["unit_buf"], w16) for _ in range(2)]
                          if self.scheme == ZERO_SCHEME_Z3 else None)
        if theta0 is not None:
            self.place_(self.master, theta0)
        self.stream = stream if stream is not None else torch.cuda.current_stream(self.device)
        self.gather_stream = gather_stream
        self.ctx = zero_init(self.scheme, self.W, self.n, self.unit_sizes, self.gdt, self.wdt, self.master,
                             self.m, self.v, self.p16, self.shard16, self.unit_bufs, self.stream, gather_stream)
        self._hook = None
        self.grad_norm = None      # fp32 scalar on the device: the last clipped step's norm
        self._clip_space = None
        zero_refresh_working_copy(self.ctx)
        self.grads = self.new_grad_buffers() if with_grad_buffers else None

    # layout helpers (marshalling between the caller's n values and the padded layout)
    def real_index(self):
        torch = self.torch
        parts = [torch.arange(o, o + s, device=self.device) for o, s in zip(self.off, self.unit_sizes)]
        return torch.cat(parts) if parts else torch.zeros(0, dtype=torch.int64, device=self.device)

    def place_(self, dst, real):
        real = self.torch.as_tensor(real).to(device=dst.device, dtype=dst.dtype)
        if len(self.unit_sizes) == 1:
            dst[: self.n].copy_(real)
        else:
            pos = 0
            for o, s in zip(self.off, self.unit_sizes):
                dst[o:o + s].copy_(real[pos:pos + s])
                pos += s
        return dst

    def new_grad_buffers(self):
        return [self._alloc(self.n_pad, self.grad_torch_dtype) for _ in range(self.W)]

    def working_copy(self):
        """The full 16-bit vector in flat order (Z3: every rank's shards interleaved back)."""
        if self.scheme != ZERO_SCHEME_Z3:
            return self.p16
        out = self.torch.empty(self.n_pad, dtype=self.work_torch_dtype, device=self.device)
        for u, (o, s, o16) in enumerate(zip(self.off, self.shard, self.off16)):
            for r in range(self.W):
                out[o + r * s:o + (r + 1) * s].copy_(self.shard16[r][o16:o16 + s])
        return out

    def step(self, grads, lr, beta1, beta2, eps, t, max_norm=None):
        """One step; with ``max_norm`` the mean gradient is clipped by its global
        norm, which ``grad_norm`` holds afterwards (on the device, in stream
        order).  The first clipped step allocates the workspace for it."""
        if max_norm is None:
            zero_step(self.ctx, self.scheme, self.W, self.n, grads, lr, beta1, beta2, eps, t)
            return
        if self._clip_space is None:
            nbytes = zero_step_clipped_workspace_bytes(self.ctx)
            with _on(self.stream, self.device):
                self._clip_space = self._alloc(nbytes, self.torch.uint8)
                self.grad_norm = self._alloc(1, self.torch.float32)
        zero_step_clipped(self.ctx, self.scheme, self.W, self.n, grads, lr, beta1, beta2, eps, t, max_norm,
                          self.grad_norm, self._clip_space, self._clip_space.numel())

    def set_unit_hook(self, fn):
        self._hook = zero_set_unit_hook(self.ctx, fn)

    def set_variant(self, variant):
        zero_set_variant(self.ctx, variant)

    def set_graph(self, on=True):
        zero_set_graph(self.ctx, on)

    def set_debug(self, flags):
        zero_set_debug(self.ctx, flags)

    def stat(self, which):
        return zero_stat(self.ctx, which)

    def sync(self, timeout_ms=-1):
        zero_sync(self.ctx, timeout_ms)

    def close(self):
        if getattr(self, "ctx", None):
            zero_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class DpReplicas:
    """W literal DP replicas allocated with PyTorch on ``device``: per replica
    an fp32 master, m and v and a 16-bit working copy, n_pad values each.

    ``theta0`` (n fp32 values) is written into every replica's master; m and
    v start at zero.  Each 16-bit working copy is written by the step (it
    holds zeros before the first one).  The step and the replica check run
    in the library.  ``alloc`` as for :class:`ZeroStep`.
    """

    def __init__(self, W, n, grad_dtype="fp16", work_dtype=None, theta0=None, device="cuda", stream=None,
                 alloc=None):
        import torch
        self.torch = torch
        self.W, self.n = int(W), int(n)
        self.gdt = _DT[grad_dtype]
        self.wdt = _DT[work_dtype if work_dtype is not None else grad_dtype]
        self.n_pad = zero_buffer_sizes(ZERO_SCHEME_DP, self.W, [self.n])["n_pad"]
        self.device = torch.device(device)
        t16 = {ZERO_FP16: torch.float16, ZERO_BF16: torch.bfloat16}
        self.grad_torch_dtype, self.work_torch_dtype = t16[self.gdt], t16[self.wdt]
        need = self.W * self.n_pad * (12 + 2)
        if self.device.type == "cuda":
            free, _ = torch.cuda.mem_get_info(self.device)
            if need > free:
                raise MemoryError(f"{self.W} replicas of {self.n_pad} parameters need {need} bytes of device "
                                  f"memory; {free} are free")
        self._alloc = alloc or _zeros_on(self.device)
        self.master = [self._alloc(self.n_pad, torch.float32) for _ in range(self.W)]
        self.m = [self._alloc(self.n_pad, torch.float32) for _ in range(self.W)]
        self.v = [self._alloc(self.n_pad, torch.float32) for _ in range(self.W)]
        self.p16 = [self._alloc(self.n_pad, self.work_torch_dtype) for _ in range(self.W)]
        if theta0 is not None:
            th = torch.as_tensor(theta0).to(device=self.device, dtype=torch.float32)
            for r in range(self.W):
                self.master[r][: self.n].copy_(th)
        self.stream = stream if stream is not None else torch.cuda.current_stream(self.device)
        self._count = self._alloc(1, torch.int64)

    def new_grad_buffers(self):
        return [self._alloc(self.n_pad, self.grad_torch_dtype) for _ in range(self.W)]

    def step(self, grads, lr, beta1, beta2, eps, t):
        zero_step_dp_replicas(self.W, self.n, self.gdt, self.wdt, grads, self.master, self.m, self.v, self.p16,
                              lr, beta1, beta2, eps, t, self.stream)

    def mismatches(self) -> int:
        """Elements, over replicas 1..W-1, that differ bitwise from replica 0 (waits)."""
        zero_dp_replicas_mismatches(self.W, self.n, self.master, self.m, self.v, self.p16, self._count,
                                    self.stream)
        self.stream.synchronize()
        return int(self._count.item())


def _itemsize(dtype) -> int:
    import torch
    return torch.empty(0, dtype=dtype).element_size()


def _round4k(nbytes: int) -> int:
    return -(-int(nbytes) // 4096) * 4096


class ZeroOffload:
    """ZeRO-2 with the optimizer on the host: fp32 master, m and v in host
    memory (the 16-bit working copy and the gradients on ``device``), the
    fp32 means and 16-bit results crossing the link through page-locked
    buffers from ``zero_host_alloc``.  ``theta0`` (n values) seeds the
    master; the device working copy is written by each step.  ``alloc`` as
    for :class:`ZeroStep`; ``host_alloc(numel, dtype)``, if given, supplies
    the five host buffers (zero-filled CPU tensors, best page-locked)
    instead of ``zero_host_alloc``."""

    def __init__(self, W, n, grad_dtype="fp16", work_dtype=None, theta0=None, device="cuda", stream=None,
                 chunk_elems=0, threads=0, alloc=None, host_alloc=None):
        import torch
        self.torch = torch
        self.W, self.n = int(W), int(n)
        self.gdt = _DT[grad_dtype]
        self.wdt = _DT[work_dtype if work_dtype is not None else grad_dtype]
        self.n_pad = zero_buffer_sizes(ZERO_SCHEME_Z2, self.W, [self.n])["n_pad"]
        self.device = torch.device(device)
        t16 = {ZERO_FP16: torch.float16, ZERO_BF16: torch.bfloat16}
        self.grad_torch_dtype, self.work_torch_dtype = t16[self.gdt], t16[self.wdt]
        self._bufs = []
        specs = [(self.n_pad, torch.float32)] * 4 + [(self.n_pad, self.work_torch_dtype)]
        if host_alloc is None:
            # one zero_host_alloc block for all five: each vector alone can be
            # smaller than a huge page, and such blocks stay on base pages, over
            # which the host pass and the link copies both measured slower
            block = HostBuffer(max(1, sum(_round4k(numel * _itemsize(d)) for numel, d in specs)), torch.uint8)
            self._bufs.append(block)
            views, pos = [], 0
            for numel, dtype in specs:
                nbytes = numel * _itemsize(dtype)
                views.append(block.tensor[pos:pos + nbytes].view(dtype))
                pos += _round4k(nbytes)
        else:
            views = [host_alloc(numel, dtype) for numel, dtype in specs]
        self.master, self.m, self.v, self.host_grad, self.host_p16 = views
        if theta0 is not None:
            self.master[: self.n].copy_(torch.as_tensor(theta0, dtype=torch.float32).cpu())
        self._alloc = alloc or _zeros_on(self.device)
        self.p16 = self._alloc(self.n_pad, self.work_torch_dtype)
        self.staging_bytes = zero_offload_staging_bytes(chunk_elems)
        self.staging = self._alloc(self.staging_bytes, torch.uint8)
        self.stream = stream if stream is not None else torch.cuda.current_stream(self.device)
        self.ctx = zero_offload_init(self.W, self.n, self.gdt, self.wdt, self.master, self.m, self.v,
                                     self.host_grad, self.host_p16, self.p16, self.staging, self.staging_bytes,
                                     chunk_elems, threads, self.stream)

    def new_grad_buffers(self):
        return [self._alloc(self.n_pad, self.grad_torch_dtype) for _ in range(self.W)]

    def step(self, grads, lr, beta1, beta2, eps, t):
        zero_offload_step(self.ctx, grads, lr, beta1, beta2, eps, t)

    def stats(self):
        return zero_offload_stats(self.ctx)

    def set_step(self, t):
        """Resume at step t: the host master, m and v must hold the state after step t."""
        zero_offload_set_step(self.ctx, t)

    def close(self):
        if getattr(self, "ctx", None):
            zero_offload_destroy(self.ctx)
            self.ctx = None
        for b in getattr(self, "_bufs", []):
            b.close()
        self._bufs = []

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---- operators of a language model around the step ----------------------------------

def _on(stream, device):
    """Allocate in the order of ``stream``, a stream or its handle (None: the current one)."""
    import contextlib

    import torch
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream(stream)
        stream = torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def _stream_getter():
    import torch
    # a tenth of a microsecond where torch.cuda.current_stream takes three
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw or (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _current_stream(index):
    """The handle of the device's current stream."""
    global _current_stream
    _current_stream = _stream_getter()
    return _current_stream(index)


def _current_device():
    """The index of the current device."""
    global _current_device
    import torch
    # without torch.cuda.current_device's check that CUDA is there
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    return _current_device()


def _rows(x, what, rows, width, dtype, device):
    """(address, row stride) of a matrix of 16-bit rows; raises ValueError where it is none."""
    shape = x.shape
    if len(shape) == 2 and shape[0] == rows and shape[1] == width and x.dtype is dtype and x.device == device:
        stride, step = x.stride()
        if step == 1 or width == 1:
            return x.data_ptr(), (stride if rows > 1 else width)
    raise ValueError(f"{what} must be a tensor on {device} of {rows} rows of {width} adjacent {dtype} values, not "
                     f"{x.dtype} {tuple(shape)} with strides {x.stride()} on {x.device}")


def _ids(x, what, device):
    """(address, bytes per id) of a contiguous vector of ids."""
    size = x.element_size()
    if size < 4 or x.is_floating_point() or x.is_complex() or not x.is_contiguous() or x.device != device:
        raise ValueError(f"{what} must be a contiguous tensor of int32 or int64 ids on {device}, not {x.dtype} on "
                         f"{x.device}")
    return x.data_ptr(), size


class _Owner:
    """What the owners below share: the format, the workspace, the stream."""

    def _setup(self, dtype, device, stream, alloc):
        import torch
        self.torch = torch
        self.dtype = _DT[dtype]
        self.torch_dtype = {ZERO_FP16: torch.float16, ZERO_BF16: torch.bfloat16}[self.dtype]
        self.device = torch.device(device)
        self.stream = stream
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device() if torch.cuda.is_available() else 0)
        self._index, self._new, self._fp32 = self.device.index, torch.empty, torch.float32
        self._alloc = alloc

    def _bind(self, name):
        """The C entry point under the owner's device, raising like its wrapper:
        the owners' calls are short enough for the wrapper's own conversions to count."""
        fn, index, torch = getattr(lib(), name), self._index, self.torch

        def call(*args):
            if _current_device() == index:
                rc = fn(*args)
            else:
                with torch.cuda.device(index):
                    rc = fn(*args)
            if rc < 0:
                raise ZeroError(rc, name, lib().zero_last_error().decode())
        return call

    def _workspace(self, nbytes, zero=0):
        """The workspace, from ``alloc`` or PyTorch with any contents; its first ``zero`` bytes are set to 0."""
        torch = self.torch
        with _on(self.stream, self.device):
            if self._alloc is not None:
                self.workspace = self._alloc(max(256, nbytes), torch.uint8)
            else:
                self.workspace = torch.empty(max(256, nbytes), dtype=torch.uint8, device=self.device)
            if zero:
                self.workspace[:zero].zero_()
        self.workspace_bytes = self.workspace.numel()
        self._ws = self.workspace.data_ptr()
        # where the workspace was used last: its fill, so far
        self._used = torch.cuda.current_stream(self.device) if self.stream is None and self.workspace.is_cuda else None
        self._used_raw = self._used.cuda_stream if self._used else None

    def _raw_stream(self, workspace=True):
        """The handle of the stream for a call, which uses the workspace or not."""
        if self.stream is not None:
            return _stream(self.stream)
        raw = _current_stream(self._index)
        if workspace and raw != self._used_raw:
            self._change_stream(raw)
        return raw or None

    def _change_stream(self, raw):
        """The workspace goes to another stream: after the work of the one that had it, and the allocator must not
        hand it out again before this one's.  A capture begins with everything before it done and its replays are
        ordered by the caller, so nothing is recorded there."""
        torch = self.torch
        with torch.cuda.device(self._index):
            if torch.cuda.is_current_stream_capturing():
                return
        here = torch.cuda.current_stream(self.device)
        here.wait_stream(self._used)
        self.workspace.record_stream(here)
        self._used, self._used_raw = here, raw

    def _empty(self, shape, dtype):
        if self.stream is None:
            return self._new(shape, dtype=dtype, device=self.device)
        with _on(self.stream, self.device):
            return self._new(shape, dtype=dtype, device=self.device)

    def _check_tokens(self, count):
        if count > self.max_tokens:
            raise ValueError(f"{count} tokens: this owner was made for up to {self.max_tokens}")


class LmLoss(_Owner):
    """Cross entropy of a head of ``vocab`` rows of ``width`` values, and its
    gradients, for up to ``max_tokens`` tokens a call (zero_lm_loss,
    zero_lm_loss_grad).  The owner holds the workspace: calls that may overlap
    on the GPU need an owner each.  Work goes to ``stream``, or to the stream
    that is current at the call; a call on another stream than the last one's
    waits for that one (a captured call does not: what a graph's replays may
    overlap is the caller's to order)."""

    def __init__(self, vocab, width, dtype="fp16", max_tokens=8192, with_grad=True, device="cuda", stream=None,
                 alloc=None):
        self._setup(dtype, device, stream, alloc)
        self.vocab, self.width, self.max_tokens = int(vocab), int(width), int(max_tokens)
        self.with_grad = bool(with_grad)
        self._workspace(zero_lm_workspace_bytes(self.max_tokens, self.vocab, self.width, self.with_grad), zero=4)
        self._loss, self._grad = self._bind("zero_lm_loss"), self._bind("zero_lm_loss_grad")
        self._status = self._bind("zero_lm_workspace_status")

    def loss(self, hidden, table, targets, loss=None, lse=None):
        """(loss, lse) of each token, fp32; loss is 0 where the target lies outside the vocabulary."""
        tokens = targets.numel()
        self._check_tokens(tokens)
        h, hs = _rows(hidden, "hidden", tokens, self.width, self.torch_dtype, self.device)
        t, ts = _rows(table, "table", self.vocab, self.width, self.torch_dtype, self.device)
        ids, id_bytes = _ids(targets, "targets", self.device)
        loss = self._empty(tokens, self._fp32) if loss is None else self._vector(loss, tokens)
        lse = self._empty(tokens, self._fp32) if lse is None else self._vector(lse, tokens)
        self._loss(tokens, self.vocab, self.width, self.dtype, h, hs, t, ts, ids, id_bytes, loss.data_ptr(),
                   lse.data_ptr(), self._ws, self.workspace_bytes, self._raw_stream())
        return loss, lse

    def grad(self, hidden, table, targets, lse, scale, dhidden=None, dtable=None, accumulate=False):
        """(dhidden, dtable) of scale * loss.sum(); with ``accumulate`` added onto the given dtable."""
        if not self.with_grad:
            raise ValueError("this owner was made without room for the gradient (with_grad=False)")
        if accumulate and dtable is None:
            raise ValueError("accumulate needs the dtable to add to")
        tokens = targets.numel()
        self._check_tokens(tokens)
        h, hs = _rows(hidden, "hidden", tokens, self.width, self.torch_dtype, self.device)
        t, ts = _rows(table, "table", self.vocab, self.width, self.torch_dtype, self.device)
        ids, id_bytes = _ids(targets, "targets", self.device)
        self._vector(lse, tokens)
        if dhidden is None:
            dhidden = self._empty((tokens, self.width), self.torch_dtype)
            dh, dhs = dhidden.data_ptr(), self.width
        else:
            dh, dhs = _rows(dhidden, "dhidden", tokens, self.width, self.torch_dtype, self.device)
        if dtable is None:
            dtable = self._empty((self.vocab, self.width), self.torch_dtype)
            dt, dts = dtable.data_ptr(), self.width
        else:
            dt, dts = _rows(dtable, "dtable", self.vocab, self.width, self.torch_dtype, self.device)
        self._grad(tokens, self.vocab, self.width, self.dtype, h, hs, t, ts, ids, id_bytes, lse.data_ptr(), scale, dh,
                   dhs, dt, dts, 1 if accumulate else 0, self._ws, self.workspace_bytes, self._raw_stream())
        return dhidden, dtable

    def _vector(self, x, tokens):
        if x.dtype != self._fp32 or x.numel() != tokens or not x.is_contiguous() or x.device != self.device:
            raise ValueError(f"loss and lse must be contiguous tensors of {tokens} fp32 values on {self.device}")
        return x

    def status(self):
        """Wait for the owner's calls so far; raises ZeroError if a device wait of theirs gave up."""
        self._status(self._ws, self._raw_stream())


class LmLogprobs(_Owner):
    """Log probabilities of given tokens under a head of ``vocab`` rows of
    ``width`` values, with the entropy of each distribution and its ``top``
    likeliest alternatives (0..16), and their gradients, for up to
    ``max_tokens`` tokens a call (zero_lm_logprobs, zero_lm_logprobs_grad).
    ``scale`` multiplies the logits: 1 / temperature.  Workspace and stream as
    for :class:`LmLoss`."""

    def __init__(self, vocab, width, dtype="fp16", max_tokens=8192, scale=1.0, top=0, with_grad=True, device="cuda",
                 stream=None, alloc=None):
        self._setup(dtype, device, stream, alloc)
        self.vocab, self.width, self.max_tokens = int(vocab), int(width), int(max_tokens)
        self.scale, self.top, self.with_grad = float(scale), int(top), bool(with_grad)
        self._workspace(zero_lm_logprobs_workspace_bytes(self.max_tokens, self.vocab, self.width, self.top,
                                                         self.with_grad), zero=4)
        self._logprobs, self._grad = self._bind("zero_lm_logprobs"), self._bind("zero_lm_logprobs_grad")
        self._status = self._bind("zero_lm_workspace_status")

    def _operands(self, hidden, table, targets):
        tokens = targets.numel()
        self._check_tokens(tokens)
        h, hs = _rows(hidden, "hidden", tokens, self.width, self.torch_dtype, self.device)
        t, ts = _rows(table, "table", self.vocab, self.width, self.torch_dtype, self.device)
        ids, id_bytes = _ids(targets, "targets", self.device)
        return tokens, (tokens, self.vocab, self.width, self.dtype, h, hs, t, ts, ids, id_bytes, self.scale)

    def logprobs(self, hidden, table, targets):
        """(logp, entropy, lse) of each token, fp32; with ``top`` also the alternatives' log probabilities and ids
        (tokens x top, fp32 and int32, the likeliest first).  logp is 0 where the target lies outside the vocabulary."""
        tokens, operands = self._operands(hidden, table, targets)
        logp, entropy, lse = self._empty(tokens, self._fp32), self._empty(tokens, self._fp32), self._empty(tokens, self._fp32)
        outs, top_logp, top_ids = (logp, entropy, lse), None, None
        if self.top:
            values, ids = self._empty((tokens, self.top), self._fp32), self._empty((tokens, self.top), self.torch.int32)
            outs, top_logp, top_ids = outs + (values, ids), values.data_ptr(), ids.data_ptr()
        self._logprobs(*operands, self.top, logp.data_ptr(), entropy.data_ptr(), lse.data_ptr(), top_logp, top_ids,
                       self._ws, self.workspace_bytes, self._raw_stream())
        return outs

    def grad(self, hidden, table, targets, lse, dlogp, entropy=None, dentropy=None, dhidden=None, dtable=None,
             accumulate=False):
        """(dhidden, dtable) from the gradients of the tokens' logp and, with ``dentropy``, of their entropy; lse and
        entropy as :meth:`logprobs` returned them.  With ``accumulate`` added onto the given dtable."""
        if not self.with_grad:
            raise ValueError("this owner was made without room for the gradient (with_grad=False)")
        if accumulate and dtable is None:
            raise ValueError("accumulate needs the dtable to add to")
        if dentropy is not None and entropy is None:
            raise ValueError("dentropy needs the entropy")
        tokens, operands = self._operands(hidden, table, targets)
        given = [None if x is None else self._vector(x, what, tokens).data_ptr()
                 for x, what in ((lse, "lse"), (dlogp, "dlogp"), (entropy, "entropy"), (dentropy, "dentropy"))]
        if dhidden is None:
            dhidden = self._empty((tokens, self.width), self.torch_dtype)
        if dtable is None:
            dtable = self._empty((self.vocab, self.width), self.torch_dtype)
        dh, dhs = _rows(dhidden, "dhidden", tokens, self.width, self.torch_dtype, self.device)
        dt, dts = _rows(dtable, "dtable", self.vocab, self.width, self.torch_dtype, self.device)
        self._grad(*operands, *given, dh, dhs, dt, dts, 1 if accumulate else 0, self._ws, self.workspace_bytes,
                   self._raw_stream())
        return dhidden, dtable

    def _vector(self, x, what, tokens):
        if x.dtype != self._fp32 or x.numel() != tokens or not x.is_contiguous() or x.device != self.device:
            raise ValueError(f"{what} must be a contiguous tensor of {tokens} fp32 values on {self.device}")
        return x

    def status(self):
        """Wait for the owner's calls so far; raises ZeroError if a device wait of theirs gave up."""
        self._status(self._ws, self._raw_stream())


class Embedding(_Owner):
    """Lookup in a table of ``vocab`` rows of ``width`` values, times ``scale``,
    and the table's gradient (zero_embedding, zero_embedding_grad), for up to
    ``max_tokens`` ids a call.  Workspace and stream as for :class:`LmLoss`."""

    def __init__(self, vocab, width, dtype="fp16", max_tokens=8192, scale=1.0, device="cuda", stream=None, alloc=None):
        self._setup(dtype, device, stream, alloc)
        self.vocab, self.width, self.max_tokens = int(vocab), int(width), int(max_tokens)
        self.scale = float(scale)
        self._workspace(zero_embedding_workspace_bytes(self.max_tokens, self.width))
        self._lookup, self._grad = self._bind("zero_embedding"), self._bind("zero_embedding_grad")

    def forward(self, tokens, table, out=None):
        """scale * table[tokens], one row per id (0 for an id outside the table)."""
        count = tokens.numel()
        t, ts = _rows(table, "table", self.vocab, self.width, self.torch_dtype, self.device)
        ids, id_bytes = _ids(tokens, "tokens", self.device)
        if out is None:
            out = self._empty((count, self.width), self.torch_dtype)
            o, os_ = out.data_ptr(), self.width
        else:
            o, os_ = _rows(out, "out", count, self.width, self.torch_dtype, self.device)
        self._lookup(count, self.vocab, self.width, self.dtype, ids, id_bytes, t, ts, self.scale, o, os_,
                     self._raw_stream(workspace=False))
        return out

    def grad(self, tokens, dout, dtable=None, accumulate=False):
        """The table's gradient, written to (or, with ``accumulate``, added onto) dtable."""
        if accumulate and dtable is None:
            raise ValueError("accumulate needs the dtable to add to")
        count = tokens.numel()
        self._check_tokens(count)
        ids, id_bytes = _ids(tokens, "tokens", self.device)
        d, ds = _rows(dout, "dout", count, self.width, self.torch_dtype, self.device)
        if dtable is None:
            dtable = self._empty((self.vocab, self.width), self.torch_dtype)
            t, ts = dtable.data_ptr(), self.width
        else:
            t, ts = _rows(dtable, "dtable", self.vocab, self.width, self.torch_dtype, self.device)
        self._grad(count, self.vocab, self.width, self.dtype, ids, id_bytes, d, ds, self.scale, t, ts,
                   1 if accumulate else 0, self._ws, self.workspace_bytes, self._raw_stream())
        return dtable


class GradClip(_Owner):
    """The global norm of the mean gradient of W ranks over tensors of the given
    element counts, and the clipped mean gradient as one flat vector, tensor
    after tensor (zero_grad_norm, zero_grad_clip).  ``grads`` is a list of W
    lists of tensors; dtype "fp16", "bf16" or "fp32"."""

    def __init__(self, numels, W=1, dtype="fp16", device="cuda", stream=None, alloc=None):
        import torch
        fp32 = dtype in ("fp32", ZERO_FP32)
        self._setup("fp16" if fp32 else dtype, device, stream, alloc)
        if fp32:
            self.dtype, self.torch_dtype = ZERO_FP32, torch.float32
        self.W = int(W)
        self.numels = [int(k) for k in numels]
        self.n = sum(self.numels)
        self._sizes, self._sizes_at = _u64_array(self.numels)
        self._expected = self.numels * self.W
        self._item = _itemsize(self.torch_dtype)
        offsets, at = [], 0
        for k in self.numels:
            offsets.append(at * self._item)
            at += k
        self._offsets = offsets
        nbytes = zero_grad_norm_workspace_bytes()
        self._workspace(nbytes, zero=nbytes)
        self._c_norm, self._c_clip = self._bind("zero_grad_norm"), self._bind("zero_grad_clip")

    def _pointers(self, grads):
        T, count = self.torch.Tensor, len(self.numels)
        flat = [g for rank in grads for g in rank]
        if (len(grads) != self.W or any(len(rank) != count for rank in grads)
                or list(map(T.numel, flat)) != self._expected):
            raise ValueError(f"grads must be {self.W} lists of tensors of the owner's sizes")
        # get_device: the index where the tensor is on a GPU (comparing devices takes three times as long)
        if ({g.dtype for g in flat} - {self.torch_dtype} or set(map(T.get_device, flat)) - {self._index}
                or not all(map(T.is_contiguous, flat))):
            raise ValueError(f"gradients must be contiguous, {self.torch_dtype} and on {self.device}")
        return _u64_array(map(T.data_ptr, flat))

    def _norm(self, ptrs_at, stream):
        norm = self._empty(1, self.torch.float32)
        self._c_norm(self.W, len(self.numels), self._sizes_at, self.dtype, ptrs_at, norm.data_ptr(), self._ws,
                     self.workspace_bytes, stream)
        return norm

    def _out(self, out):
        if out is None:
            return self._empty(self.n, self.torch_dtype)
        if (out.numel() != self.n or out.dtype != self.torch_dtype or not out.is_contiguous()
                or out.device != self.device):
            raise ValueError(f"out must be {self.n} contiguous values of {self.torch_dtype} on {self.device}")
        return out

    def _clip(self, ptrs_at, norm, max_norm, out, stream):
        base = out.data_ptr()
        outs, outs_at = _u64_array([base + o for o in self._offsets])
        self._c_clip(self.W, len(self.numels), self._sizes_at, self.dtype, ptrs_at, norm.data_ptr(), max_norm, outs_at,
                     stream)
        return out

    def norm(self, grads):
        """The norm, one fp32 value on the device."""
        ptrs, at = self._pointers(grads)
        return self._norm(at, self._raw_stream())

    def clip(self, grads, norm, max_norm, out=None):
        """The flat mean gradient times min(1, max_norm / (norm + 1e-6))."""
        if norm.dtype != self._fp32 or norm.numel() != 1 or norm.device != self.device:
            raise ValueError(f"norm must be one fp32 value on {self.device}, not {norm.dtype} {tuple(norm.shape)} on "
                             f"{norm.device}")
        ptrs, at = self._pointers(grads)
        return self._clip(at, norm, max_norm, self._out(out), self._raw_stream(workspace=False))

    def norm_and_clip(self, grads, max_norm, out=None):
        """(norm, flat clipped mean gradient)."""
        ptrs, at = self._pointers(grads)
        out, stream = self._out(out), self._raw_stream()
        norm = self._norm(at, stream)
        return norm, self._clip(at, norm, max_norm, out, stream)


def _starts(shapes):
    """Where each matrix starts in a flat vector, on boundaries of 8 values, and the vector's length."""
    at, starts = 0, []
    for r, c in shapes:
        starts.append(at)
        at += -(-r * c // 8) * 8
    return starts, at


class _Matrices(_Owner):
    """What the owners over a list of matrices share."""

    def _setup_matrices(self, shapes, coefficients, fine_steps):
        self.shapes = [(int(r), int(c)) for r, c in shapes]
        self.starts, self.n = _starts(self.shapes)
        self._keep, self._rows_at, self._cols_at = _shape_arrays(self.shapes)
        self.steps, self._co, self._co_at = _steps_of(coefficients)
        self.fine_steps = -1 if fine_steps is None else int(fine_steps)

    def views(self, flat):
        """The matrices in a flat vector laid out like the owner's."""
        return [flat[at:at + r * c].view(r, c) for (r, c), at in zip(self.shapes, self.starts)]

    def status(self):
        """Wait for the owner's calls so far; raises ZeroError if a device wait of theirs gave up."""
        self._status(self._ws, self._raw_stream())


class Orthogonalize(_Matrices):
    """Newton-Schulz orthogonalisation of matrices of the given (rows, cols),
    all of one dtype: "fp16", "bf16" or "fp32" (zero_orthogonalize).
    ``coefficients`` holds (a, b, c) for each step; ``fine_steps`` of them carry
    their operands in two 16-bit parts (None: all, for bf16 all but the last).  Workspace and stream as for :class:`LmLoss`."""

    def __init__(self, shapes, dtype="bf16", coefficients=MUON_COEFFICIENTS, fine_steps=None, device="cuda",
                 stream=None, alloc=None):
        import torch
        fp32 = dtype in ("fp32", ZERO_FP32)
        self._setup("fp16" if fp32 else dtype, device, stream, alloc)
        if fp32:
            self.dtype, self.torch_dtype = ZERO_FP32, torch.float32
        self._setup_matrices(shapes, coefficients, fine_steps)
        self._workspace(zero_orthogonalize_workspace_bytes(self.shapes), zero=4)
        self._call, self._status = self._bind("zero_orthogonalize"), self._bind("zero_lm_workspace_status")

    def _addresses(self, matrices, what):
        if len(matrices) != len(self.shapes):
            raise ValueError(f"{what}: {len(matrices)} matrices, this owner was made for {len(self.shapes)}")
        both = [_rows(x, what, r, c, self.torch_dtype, self.device) for x, (r, c) in zip(matrices, self.shapes)]
        return _u64_array([a for a, _ in both]), _u64_array([s for _, s in both])

    def forward(self, matrices, out=None):
        """The orthogonalised matrices, written to ``out`` (which may be the matrices themselves) or to new memory."""
        (ins, ins_at), (si, si_at) = self._addresses(matrices, "matrices")
        if out is None:
            out = [self._empty(s, self.torch_dtype) for s in self.shapes]
        (outs, outs_at), (so, so_at) = self._addresses(out, "out")
        self._call(len(self.shapes), self._rows_at, self._cols_at, self.dtype, ins_at, si_at, outs_at, so_at,
                   self.steps, self._co_at, self.fine_steps, self._ws, self.workspace_bytes, self._raw_stream())
        return out


class MuonStep(_Matrices):
    """The step of W ranks on matrices of the given (rows, cols) that takes its
    direction from the orthogonalised momentum (zero_muon_step).  ``master``,
    ``momentum`` (fp32) and ``p16`` are flat vectors, matrix after matrix, each
    starting on a boundary of 8 values (``views`` cuts them up); ``theta0``, a
    list of matrices, seeds the master and the 16-bit copy.  ``scales``
    multiplies the learning rate of each matrix (None: 1); ``fine_steps`` is as
    for :class:`Orthogonalize` (None: all).  What a ZeRO step trains beside them
    (embeddings, vectors) has a :class:`ZeroStep` of its own.
    ``alloc`` as for :class:`ZeroStep`; workspace and stream as for
    :class:`LmLoss`."""

    def __init__(self, shapes, W=1, grad_dtype="fp16", work_dtype=None, theta0=None, coefficients=MUON_COEFFICIENTS,
                 fine_steps=None, scales=None, device="cuda", stream=None, alloc=None):
        import torch
        self._setup(grad_dtype, device, stream, alloc)
        self.W = int(W)
        self.wdt = _DT[work_dtype if work_dtype is not None else grad_dtype]
        self._setup_matrices(shapes, coefficients, fine_steps)
        if scales is not None and len(scales) != len(self.shapes):
            raise ValueError(f"scales must hold one factor for each of the {len(self.shapes)} matrices")
        if theta0 is not None:
            theta0 = [torch.as_tensor(x) for x in theta0]
            if [tuple(x.shape) for x in theta0] != self.shapes:
                raise ValueError("theta0 must be a list of matrices of the owner's shapes")
        self.scales = None if scales is None else [float(x) for x in scales]
        self._sc, self._sc_at = (None, None) if scales is None else _c_array("d", self.scales)
        self._workspace(zero_muon_workspace_bytes(self.W, self.shapes), zero=4)
        new = alloc or _zeros_on(self.device)
        work = {ZERO_FP16: torch.float16, ZERO_BF16: torch.bfloat16}[self.wdt]
        with _on(self.stream, self.device):
            self.master, self.momentum = new(self.n, torch.float32), new(self.n, torch.float32)
            self.p16 = new(self.n, work)
            if theta0 is not None:
                for to, x in zip(self.views(self.master), theta0):
                    to.copy_(x)
                self.p16.copy_(self.master)
        self._new_state = new
        self._state = [_u64_array([x.data_ptr() + at * x.element_size() for at in self.starts])
                       for x in (self.master, self.momentum, self.p16)]
        self._call, self._status = self._bind("zero_muon_step"), self._bind("zero_lm_workspace_status")

    def new_grad_buffers(self):
        """W lists of matrices for the ranks' gradients, each list in one flat vector."""
        with _on(self.stream, self.device):
            return [self.views(self._new_state(self.n, self.torch_dtype)) for _ in range(self.W)]

    def _change_stream(self, raw):
        super()._change_stream(raw)
        if self._used_raw == raw:
            for x in (self.master, self.momentum, self.p16):
                x.record_stream(self._used)

    def step(self, grads, lr, mu=0.95, weight_decay=0.0, nesterov=True):
        """One step; ``grads`` is W lists of contiguous matrices."""
        T = self.torch.Tensor
        flat = [g for rank in grads for g in rank]
        if (len(grads) != self.W or any(len(rank) != len(self.shapes) for rank in grads)
                or [tuple(g.shape) for g in flat] != self.shapes * self.W):
            raise ValueError(f"grads must be {self.W} lists of matrices of the owner's shapes")
        if ({g.dtype for g in flat} - {self.torch_dtype}
                or any(g.device != self.device for g in flat) or not all(map(T.is_contiguous, flat))):
            raise ValueError(f"gradients must be contiguous, {self.torch_dtype} and on {self.device}")
        ptrs, at = _u64_array(map(T.data_ptr, flat))
        self._call(self.W, len(self.shapes), self._rows_at, self._cols_at, self.dtype, self.wdt, at,
                   *(a for _, a in self._state), lr, mu, 1 if nesterov else 0, weight_decay, self._sc_at, self.steps,
                   self._co_at, self.fine_steps, self._ws, self.workspace_bytes, self._raw_stream())
