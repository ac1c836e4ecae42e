"""Thin ctypes binding of libbitdelta.so (C ABI in ``include/bitdelta.h``).

Function names match the C entry points.  This module only marshals
arguments: torch tensors become device pointers and sizes, the current torch
CUDA stream is passed as the stream, and a non-zero status raises
``BitDeltaError``.  Every step of the computation runs in the library's CUDA
kernels; there is no fallback, and a missing library is an error.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libbitdelta.so")
# the bounds-checked build (``build.build(debug=True)``): load it with load_library(LIB_DEBUG_PATH)
LIB_DEBUG_PATH = os.path.join(_HERE, "lib", "libbitdelta_debug.so")

BD_OK = 0
BD_ERR_INVALID_ARG = 1
BD_ERR_UNSUPPORTED_SHAPE = 2
BD_ERR_MISALIGNED = 3
BD_ERR_WORKSPACE = 4
BD_ERR_CUDA = 5
BD_ERR_DEVICE_TIMEOUT = 6
BD_ERR_BAD_VARIANT_ID = 7
BD_ERR_NO_SPACE = 8
BD_ERR_DEVICE_BOUNDS = 9
BD_ERR_BAD_INDEX = 10
BD_ALPHA_SCALAR = 0
BD_ALPHA_PER_ROW = 1
BD_MAX_VARIANTS = 64
BD_NOALLOC_MAX_PARTIALS = 131072
BD_LINEAR_BATCH_MAX = 256
BD_COMPRESS_BATCH_MAX = 4096
BD_COMPRESS_BATCH_PER_LAUNCH = 8
BD_LINEAR_BATCH_PER_LAUNCH = 8
BD_Y_BF16 = 0
BD_Y_E4M3 = 1
BD_KV_BF16 = 0
BD_KV_E4M3 = 1
BD_LOGITS_BF16 = 0
BD_LOGITS_F32 = 1
BD_NORM_MAX_N = 32768
BD_KV_MAX_HEADS = 1024
BD_SAMPLE_MAX_VOCAB = 262144
BD_OPT_COMPRESS_FORM = 1
BD_OPT_GROUPED_PATH = 2
BD_OPT_BATCH_KERNEL = 3
BD_OPT_BATCH_SINGLE = 4
BD_OPT_BATCH_GRID = 5
BD_OPT_TEST_STALL = 6
BD_OPT_PREFILL_KERNEL = 7
BD_OPT_PAIR_RING = 8

_lock = threading.Lock()
_lib = None


class LinearDesc(ctypes.Structure):
    """bd_linear_desc: one problem of bd_linear_batch (device pointers and sizes)."""
    _fields_ = [("x", ctypes.c_void_p), ("w_base", ctypes.c_void_p), ("bits", ctypes.c_void_p),
                ("alpha", ctypes.c_void_p), ("y", ctypes.c_void_p), ("m", ctypes.c_int64),
                ("n_out", ctypes.c_int64), ("n_in", ctypes.c_int64), ("alpha_mode", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class CompressDesc(ctypes.Structure):
    """bd_compress_desc: one matrix of bd_compress_batch (device pointers and sizes)."""
    _fields_ = [("w_base", ctypes.c_void_p), ("w_ft", ctypes.c_void_p), ("bits_out", ctypes.c_void_p),
                ("alpha_out", ctypes.c_void_p), ("n_out", ctypes.c_int64), ("n_in", ctypes.c_int64),
                ("alpha_mode", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class KVCacheDesc(ctypes.Structure):
    """bd_kv_cache: the pools of one layer's paged key-value cache (device pointers and sizes)."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32), ("kv_type", ctypes.c_int32)]


class BitDeltaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {bd_status_string(status)} (status {status})")


def load_library(path: str | None = None):
    """Open libbitdelta.so (built by ``bit_delta_tenant_gb300.build``); raises if absent."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"libbitdelta.so not found at {p}; build it with "
                               "`python -m bit_delta_tenant_gb300.build` (nvcc, sm_103a)")
        lib = ctypes.CDLL(p)
        V, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        lib.bd_version.restype = I32
        lib.bd_build_flags.restype = I32
        lib.bd_status_string.argtypes = [I32]
        lib.bd_status_string.restype = ctypes.c_char_p
        lib.bd_set_wait_limit_ns.argtypes = [I64]
        lib.bd_set_wait_limit_ns.restype = I64
        lib.bd_set_linear_path.argtypes = [I32]
        lib.bd_set_linear_path.restype = I32
        lib.bd_reconstruct.argtypes = [V, V, V, I32, I64, I64, V, V]
        lib.bd_reconstruct.restype = I32
        lib.bd_cache_state_size.argtypes = [I32]
        lib.bd_cache_state_size.restype = SZ
        lib.bd_cache_create.argtypes = [V, SZ, I32, V, SZ, ctypes.c_double, I32, ctypes.POINTER(V)]
        lib.bd_cache_create.restype = I32
        lib.bd_cache_destroy.argtypes = [V]
        lib.bd_cache_destroy.restype = I32
        lib.bd_cache_register.argtypes = [V, I32, V, SZ, V, SZ]
        lib.bd_cache_register.restype = I32
        lib.bd_cache_set_pinned.argtypes = [V, I32, I32]
        lib.bd_cache_set_pinned.restype = I32
        lib.bd_cache_acquire.argtypes = [V, I32, ctypes.c_double, V, ctypes.POINTER(V), ctypes.POINTER(V)]
        lib.bd_cache_acquire.restype = I32
        lib.bd_cache_release.argtypes = [V, I32, V]
        lib.bd_cache_release.restype = I32
        lib.bd_cache_get_stats.argtypes = [V, ctypes.POINTER(CacheStats)]
        lib.bd_cache_get_stats.restype = I32
        lib.bd_cache_is_resident.argtypes = [V, I32]
        lib.bd_cache_is_resident.restype = I32
        lib.bd_set_option.argtypes = [I32, I64]
        lib.bd_set_option.restype = I64
        lib.bd_set_weight_prefetch.argtypes = [I32]
        lib.bd_set_weight_prefetch.restype = I32
        lib.bd_get_device_status.argtypes = [V]
        lib.bd_get_device_status.restype = I32
        lib.bd_compress_workspace_size.argtypes = [I64, I64, I32]
        lib.bd_compress_workspace_size.restype = SZ
        lib.bd_compress.argtypes = [V, V, I64, I64, I32, V, V, V, SZ, V]
        lib.bd_compress.restype = I32
        lib.bd_compress_noalloc.argtypes = [V, V, I64, I64, I32, V, V, V]
        lib.bd_compress_noalloc.restype = I32
        lib.bd_linear.argtypes = [V, I64, V, V, V, I32, I64, I64, V, V]
        lib.bd_linear.restype = I32
        lib.bd_compress_batch_workspace_size.argtypes = [ctypes.POINTER(CompressDesc), I32]
        lib.bd_compress_batch_workspace_size.restype = SZ
        lib.bd_compress_batch.argtypes = [ctypes.POINTER(CompressDesc), I32, V, SZ, V]
        lib.bd_compress_batch.restype = I32
        lib.bd_linear_batch_workspace_size.argtypes = [ctypes.POINTER(LinearDesc), I32]
        lib.bd_linear_batch_workspace_size.restype = SZ
        lib.bd_linear_batch.argtypes = [ctypes.POINTER(LinearDesc), I32, V, SZ, V]
        lib.bd_linear_batch.restype = I32
        lib.bd_linear_grouped_workspace_size.argtypes = [I64, I32, I64, I64]
        lib.bd_linear_grouped_workspace_size.restype = SZ
        lib.bd_linear_grouped.argtypes = [V, V, I64, V, V, V, V, I32, I64, I64, V, V, SZ, V]
        lib.bd_linear_grouped.restype = I32
        F32, CACHE = ctypes.c_float, ctypes.POINTER(KVCacheDesc)
        lib.bd_rmsnorm.argtypes = [V, V, V, V, I32, I64, I64, F32, V, I32, V, I32, V, V]
        lib.bd_rmsnorm.restype = I32
        lib.bd_kv_append.argtypes = [CACHE, V, I32, V, V, I64, V, V, V, I32, I32, V, I64, V, V]
        lib.bd_kv_append.restype = I32
        lib.bd_kv_read.argtypes = [CACHE, V, I32, I32, V, I64, V, V, V]
        lib.bd_kv_read.restype = I32
        lib.bd_attention_workspace_size.argtypes = [CACHE, I32, I32]
        lib.bd_attention_workspace_size.restype = SZ
        lib.bd_attention_decode.argtypes = [CACHE, V, I32, V, V, I32, I32, F32, I32, V, V, V, SZ, V]
        lib.bd_attention_decode.restype = I32
        lib.bd_sample.argtypes = [V, I32, I64, I64, V, V, V, V, V, V, V, V]
        lib.bd_sample.restype = I32
        _lib = lib
        return lib


def _stream(stream=None) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream if hasattr(s, "cuda_stream") else int(s))


_NOT_ON_DEVICE = "tensors passed to libbitdelta must be on a CUDA device"


def _address(t: torch.Tensor) -> int:
    """Address of a contiguous tensor in device memory: the kernels read it without further checks."""
    if not t.is_contiguous():
        raise ValueError("tensors passed to libbitdelta must be contiguous")
    if not t.is_cuda:
        raise ValueError(_NOT_ON_DEVICE)
    return t.data_ptr()


def _ptr(t: torch.Tensor | None) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else _address(t))


def _host_ptr(t: torch.Tensor) -> ctypes.c_void_p:
    """Address of a contiguous tensor that the library reads or writes from the host or by copies."""
    if not t.is_contiguous():
        raise ValueError("tensors passed to libbitdelta must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _check(rc: int, where: str) -> None:
    if rc != BD_OK:
        raise BitDeltaError(rc, where)


def bd_version() -> int:
    return int(load_library().bd_version())


def bd_build_flags() -> int:
    return int(load_library().bd_build_flags())


def bd_status_string(status: int) -> str:
    return load_library().bd_status_string(int(status)).decode()


def bd_set_wait_limit_ns(limit_ns: int) -> int:
    return int(load_library().bd_set_wait_limit_ns(int(limit_ns)))


def bd_set_linear_path(path: int) -> int:
    return int(load_library().bd_set_linear_path(int(path)))


def bd_set_option(option: int, value: int) -> int:
    """Force one kernel choice (BD_OPT_*); returns the previous value, -1 if rejected."""
    return int(load_library().bd_set_option(int(option), int(value)))


class option:
    """Context manager: bd_set_option(opt, value) inside, the previous value restored after."""

    def __init__(self, opt: int, value: int):
        self.opt, self.value = opt, value

    def __enter__(self):
        self.prev = bd_set_option(self.opt, self.value)
        if self.prev < 0:
            raise ValueError(f"bd_set_option({self.opt}, {self.value}) rejected")
        return self

    def __exit__(self, *exc):
        bd_set_option(self.opt, self.prev)


class CacheStats(ctypes.Structure):
    _fields_ = [("acquires", ctypes.c_int64), ("hits", ctypes.c_int64), ("misses", ctypes.c_int64),
                ("joined", ctypes.c_int64), ("loads", ctypes.c_int64), ("evictions", ctypes.c_int64),
                ("bytes_loaded", ctypes.c_int64), ("resident_bytes", ctypes.c_int64),
                ("resident", ctypes.c_int32), ("in_use", ctypes.c_int32)]


class DeltaCache:
    """Thin owner of a bd_cache: the state buffer (host), the arena (a torch
    tensor on the device, or a host tensor with host_arena=True) and the host
    deltas it registers are kept alive here; every call is the C entry point."""

    def __init__(self, max_variants: int, arena: torch.Tensor, half_life_s: float = 10.0, host_arena: bool = False):
        lib = load_library()
        size = lib.bd_cache_state_size(int(max_variants))
        if size == 0:
            raise ValueError("max_variants out of range")
        self._state = ctypes.create_string_buffer(size)
        self._arena = arena
        self._keep = {}
        self._handle = ctypes.c_void_p()
        self._host = bool(host_arena)
        rc = lib.bd_cache_create(ctypes.addressof(self._state), size, int(max_variants),
                                 _host_ptr(arena) if host_arena else _ptr(arena),
                                 arena.numel() * arena.element_size(), float(half_life_s), 1 if host_arena else 0,
                                 ctypes.byref(self._handle))
        _check(rc, "bd_cache_create")

    def register(self, variant: int, bits: torch.Tensor, alpha: torch.Tensor) -> None:
        rc = load_library().bd_cache_register(self._handle, int(variant), _host_ptr(bits), bits.numel(), _host_ptr(alpha),
                                              alpha.numel() * 4)
        _check(rc, "bd_cache_register")
        self._keep[variant] = (bits, alpha)

    def set_pinned(self, variant: int, pinned: bool) -> None:
        _check(load_library().bd_cache_set_pinned(self._handle, int(variant), 1 if pinned else 0), "bd_cache_set_pinned")

    def acquire(self, variant: int, now_s: float = -1.0, stream=None):
        """(status, bits_ptr, alpha_ptr) -- raw device (or arena) addresses."""
        b, a = ctypes.c_void_p(), ctypes.c_void_p()
        rc = load_library().bd_cache_acquire(self._handle, int(variant), float(now_s), self._s(stream),
                                             ctypes.byref(b), ctypes.byref(a))
        return int(rc), b.value or 0, a.value or 0

    def release(self, variant: int, stream=None) -> int:
        return int(load_library().bd_cache_release(self._handle, int(variant), self._s(stream)))

    def _s(self, stream):
        return ctypes.c_void_p(0) if self._host else _stream(stream)

    def stats(self) -> CacheStats:
        st = CacheStats()
        _check(load_library().bd_cache_get_stats(self._handle, ctypes.byref(st)), "bd_cache_get_stats")
        return st

    def is_resident(self, variant: int) -> bool:
        return bool(load_library().bd_cache_is_resident(self._handle, int(variant)))

    def close(self) -> None:
        if self._handle:
            _check(load_library().bd_cache_destroy(self._handle), "bd_cache_destroy")
            self._handle = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def bd_set_weight_prefetch(enable: int) -> int:
    return int(load_library().bd_set_weight_prefetch(int(enable)))


def bd_get_device_status(stream=None) -> int:
    return int(load_library().bd_get_device_status(_stream(stream)))


def bd_compress_workspace_size(n_out: int, n_in: int, alpha_mode: int) -> int:
    return int(load_library().bd_compress_workspace_size(n_out, n_in, alpha_mode))


def bd_compress(w_base: torch.Tensor, w_ft: torch.Tensor, alpha_mode: int, bits_out: torch.Tensor,
                alpha_out: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    """Packed sign bits and alpha of (W_base, W_ft); all tensors on the device."""
    n_out, n_in = w_base.shape
    rc = load_library().bd_compress(_ptr(w_base), _ptr(w_ft), n_out, n_in, int(alpha_mode), _ptr(bits_out),
                                    _ptr(alpha_out), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                    _stream(stream))
    _check(rc, "bd_compress")


def bd_compress_noalloc(w_base: torch.Tensor, w_ft: torch.Tensor, alpha_mode: int, bits_out: torch.Tensor,
                        alpha_out: torch.Tensor, stream=None) -> None:
    """bd_compress without a workspace, for callers that cannot allocate device memory.

    Uses the library's built-in 1 MiB scratch array; shapes needing more partial
    sums than BD_NOALLOC_MAX_PARTIALS raise (status BD_ERR_WORKSPACE).  Calls
    that overlap on the GPU share that array and race: keep them ordered.
    """
    n_out, n_in = w_base.shape
    rc = load_library().bd_compress_noalloc(_ptr(w_base), _ptr(w_ft), n_out, n_in, int(alpha_mode),
                                            _ptr(bits_out), _ptr(alpha_out), _stream(stream))
    _check(rc, "bd_compress_noalloc")


def bd_linear(x: torch.Tensor, w_base: torch.Tensor, bits: torch.Tensor, alpha: torch.Tensor, alpha_mode: int,
              y: torch.Tensor, stream=None) -> None:
    """y[m, n_out] = x[m, n_in] . (W_base + alpha * sign)^T."""
    m = x.shape[0] if x.dim() == 2 else 0
    n_out, n_in = w_base.shape
    rc = load_library().bd_linear(_ptr(x), m, _ptr(w_base), _ptr(bits), _ptr(alpha), int(alpha_mode), n_out, n_in,
                                  _ptr(y), _stream(stream))
    _check(rc, "bd_linear")


def compress_descs(problems) -> ctypes.Array:
    """bd_compress_desc array from (w_base, w_ft, alpha_mode, bits_out, alpha_out) tuples of tensors."""
    arr = (CompressDesc * len(problems))()
    for d, (w_base, w_ft, alpha_mode, bits_out, alpha_out) in zip(arr, problems):
        n_out, n_in = w_base.shape
        d.w_base, d.w_ft, d.bits_out, d.alpha_out = (_ptr(w_base).value, _ptr(w_ft).value, _ptr(bits_out).value,
                                                     _ptr(alpha_out).value)
        d.n_out, d.n_in, d.alpha_mode, d.reserved = n_out, n_in, int(alpha_mode), 0
    return arr


def bd_compress_batch_workspace_size(descs: ctypes.Array) -> int:
    return int(load_library().bd_compress_batch_workspace_size(descs, len(descs)))


def bd_compress_batch(descs: ctypes.Array, workspace: torch.Tensor, stream=None) -> None:
    """Each matrix's (bits, alpha) as bd_compress gives it, several matrices per launch."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load_library().bd_compress_batch(descs, len(descs), _ptr(workspace), ws_bytes, _stream(stream))
    _check(rc, "bd_compress_batch")


def linear_descs(problems) -> ctypes.Array:
    """bd_linear_desc array from (x, w_base, bits, alpha, alpha_mode, y) tuples of tensors."""
    arr = (LinearDesc * len(problems))()
    for d, (x, w_base, bits, alpha, alpha_mode, y) in zip(arr, problems):
        n_out, n_in = w_base.shape
        d.x, d.w_base, d.bits, d.alpha, d.y = (_ptr(x).value, _ptr(w_base).value, _ptr(bits).value,
                                               _ptr(alpha).value, _ptr(y).value)
        d.m = x.shape[0] if x.dim() == 2 else 0
        d.n_out, d.n_in, d.alpha_mode, d.reserved = n_out, n_in, int(alpha_mode), 0
    return arr


def bd_linear_batch_workspace_size(descs: ctypes.Array) -> int:
    return int(load_library().bd_linear_batch_workspace_size(descs, len(descs)))


def bd_linear_batch(descs: ctypes.Array, workspace: torch.Tensor | None, stream=None) -> None:
    """Each problem's y = x . (W_base + alpha * sign)^T, independent problems batched per launch.

    `descs` comes from `linear_descs`; `workspace` is a zero-filled device buffer of at
    least `bd_linear_batch_workspace_size(descs)` bytes (left ready for the next call)."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load_library().bd_linear_batch(descs, len(descs), _ptr(workspace), ws_bytes, _stream(stream))
    _check(rc, "bd_linear_batch")


def bd_linear_grouped_workspace_size(m: int, n_variants: int, n_out: int, n_in: int) -> int:
    return int(load_library().bd_linear_grouped_workspace_size(m, n_variants, n_out, n_in))


def bd_reconstruct(w_base: torch.Tensor, bits: torch.Tensor, alpha: torch.Tensor, alpha_mode: int,
                   w_eff: torch.Tensor, stream=None) -> None:
    """W_eff = bf16(W_base + alpha * s), materialised (for a standard matmul)."""
    n_out, n_in = w_base.shape
    rc = load_library().bd_reconstruct(_ptr(w_base), _ptr(bits), _ptr(alpha), int(alpha_mode), n_out, n_in,
                                       _ptr(w_eff), _stream(stream))
    _check(rc, "bd_reconstruct")


def bd_linear_grouped(x: torch.Tensor, variant_ids: torch.Tensor, w_base: torch.Tensor, bits_v, alpha_v,
                      alpha_modes_v, y: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    """Multi-tenant fused linear: token t uses (bits_v[ids[t]], alpha_v[ids[t]])."""
    n_var = len(bits_v)
    if len(alpha_v) != n_var or len(alpha_modes_v) != n_var:
        raise ValueError("bits_v, alpha_v and alpha_modes_v must have one entry per variant")
    m = x.shape[0]
    n_out, n_in = w_base.shape
    bits_arr = (ctypes.c_void_p * n_var)(*[_address(b) for b in bits_v])
    alpha_arr = (ctypes.c_void_p * n_var)(*[_address(a) for a in alpha_v])
    modes_arr = (ctypes.c_int32 * n_var)(*[int(md) for md in alpha_modes_v])
    rc = load_library().bd_linear_grouped(_ptr(x), _ptr(variant_ids), m, _ptr(w_base), bits_arr, alpha_arr,
                                          modes_arr, n_var, n_out, n_in, _ptr(y), _ptr(workspace),
                                          workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, "bd_linear_grouped")


# ---- the rest of a decode step: norm, key-value cache, attention, sampling ----------------
# Tensors are checked here for type, shape, layout and device, because the library sees only their
# addresses.  A decode step makes many of these calls on small inputs, so the checks are kept to a
# few attribute reads per tensor and the stream is read as a raw handle.


def _refuse(t: torch.Tensor, name: str, shape, dtype, device) -> None:
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() < 0:
        raise ValueError(f"{name}: {_NOT_ON_DEVICE}")
    if t.get_device() != device:
        raise ValueError(f"{name}: expected a tensor on CUDA device {device}, got one on {t.get_device()}")
    raise ValueError(f"{name}: tensors passed to libbitdelta must be contiguous")


def _first(t: torch.Tensor, name: str, dtype) -> tuple[int, int]:
    """Address of a contiguous tensor of the given type, and the CUDA device on which all other tensors of its call have to be."""
    device = t.get_device()
    if device < 0 or t.dtype is not dtype or not t.is_contiguous():
        _refuse(t, name, t.shape, dtype, device)
    return t.data_ptr(), device


def _arg(t: torch.Tensor | None, name: str, shape, dtype, device: int) -> int | None:
    """Address of a contiguous tensor of the given shape and type on that device (None stays NULL)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != device:
        _refuse(t, name, shape, dtype, device)
    return t.data_ptr()


def _raw_stream(stream, device: int) -> int:
    """Handle of `stream`, or of the device's current stream."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_BF16, _E4M3, _F32, _I32, _U8 = torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.int32, torch.uint8


def bd_rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float, y: torch.Tensor, residual: torch.Tensor | None = None,
               residual_out: torch.Tensor | None = None, y_scale: torch.Tensor | None = None,
               weight_ids: torch.Tensor | None = None, stream=None) -> None:
    """y = rms-norm of x + residual, scaled by weight[weight_ids[row]] (weight is [n] or [n_weights, n]).

    `residual_out` receives bf16(x + residual) and may be `residual` itself.  A bf16 `y` is
    rounded once; a float8_e4m3fn `y` comes with `y_scale`, fp32 [m, n / 128] (a scale per
    128 columns) or [m, 1] (one per row)."""
    (xp, device), shape = _first(x, "x", _BF16), x.shape
    m, n = shape
    n_weights, w_shape = (weight.shape[0], (weight.shape[0], n)) if weight.dim() == 2 else (1, (n,))
    y_type, scale_cols, scale = BD_Y_BF16, 0, None
    if y.dtype is _E4M3:
        y_type = BD_Y_E4M3
        cols = y_scale.shape[1] if y_scale is not None and y_scale.dim() == 2 else 0
        if cols < 1 or n % cols != 0:
            raise ValueError("y_scale: an 8-bit y comes with scales of shape [m, n / 128] or [m, 1]")
        scale_cols, scale = n // cols, _arg(y_scale, "y_scale", (m, cols), _F32, device)
    elif y_scale is not None:
        raise ValueError("y_scale: only an 8-bit y has scales")
    rc = (_lib or load_library()).bd_rmsnorm(
        xp, None if residual is None else _arg(residual, "residual", shape, _BF16, device),
        _arg(weight, "weight", w_shape, _BF16, device), None if weight_ids is None else _arg(weight_ids, "weight_ids", (m,), _I32, device),
        n_weights, m, n, eps, _arg(y, "y", shape, _E4M3 if y_type else _BF16, device), y_type, scale, scale_cols,
        None if residual_out is None else _arg(residual_out, "residual_out", shape, _BF16, device), _raw_stream(stream, device))
    if rc:
        _check(rc, "bd_rmsnorm")


class KVCache:
    """The pools of one layer's paged key-value cache (bd_kv_cache); keeps the tensors alive.

    k, v: [n_pages, kv_heads, page_size, head_dim], bf16, or float8_e4m3fn with k_scale and
    v_scale, the exponent bytes of their rows' power-of-two scales, uint8 [n_pages, kv_heads,
    page_size]."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor | None = None,
                 v_scale: torch.Tensor | None = None):
        if k.dim() != 4:
            raise ValueError("k: expected [n_pages, kv_heads, page_size, head_dim]")
        if k.dtype not in (_BF16, _E4M3):
            raise ValueError(f"k: expected torch.bfloat16 or torch.float8_e4m3fn, got {k.dtype}")
        e4m3 = k.dtype == _E4M3
        if e4m3 != (k_scale is not None) or e4m3 != (v_scale is not None):
            raise ValueError("k_scale and v_scale come with an 8-bit cache, and only with one")
        n_pages, self.kv_heads, self.page_size, self.head_dim = k.shape
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        d = self.desc = KVCacheDesc()
        d.k, device = _first(k, "k", k.dtype)
        self.device = device
        d.v = _arg(v, "v", k.shape, k.dtype, device)
        d.k_scale = _arg(k_scale, "k_scale", k.shape[:3], _U8, device)
        d.v_scale = _arg(v_scale, "v_scale", k.shape[:3], _U8, device)
        d.n_pages, d.kv_heads, d.head_dim, d.page_size = n_pages, self.kv_heads, self.head_dim, self.page_size
        d.kv_type = BD_KV_E4M3 if e4m3 else BD_KV_BF16
        self._ref = ctypes.byref(d)


def _table(page_table: torch.Tensor, device: int):
    """(address, n_seqs, max_pages) of a page table."""
    shape = page_table.shape
    if len(shape) != 2:
        raise ValueError("page_table: expected [n_seqs, max_pages]")
    return _arg(page_table, "page_table", shape, _I32, device), shape[0], shape[1]


def bd_kv_append(cache: KVCache, q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
                 page_table: torch.Tensor, rope: torch.Tensor | None, q_out: torch.Tensor | None,
                 seq_ids: torch.Tensor | None = None, stream=None) -> None:
    """Rotate q [t, q_heads, head_dim] into q_out and k [t, kv_heads, head_dim]; write k and v to the cache.

    Token i goes to position positions[i] of sequence seq_ids[i] (of sequence i without
    seq_ids); a negative position skips it.  `rope` is fp32 [positions, head_dim], cosines then
    sines; without it nothing is rotated and q and q_out are None.  q_out may be q."""
    n, dim, device = k.shape[0], cache.head_dim, cache.device
    kv_shape = (n, cache.kv_heads, dim)
    q_heads, qp, qo = 0, None, None
    if q is not None or q_out is not None:
        if q is None or q_out is None or q.dim() != 3:
            raise ValueError("q, q_out: both [tokens, q_heads, head_dim], or neither")
        q_heads = q.shape[1]
        qp, qo = _arg(q, "q", (n, q_heads, dim), _BF16, device), _arg(q_out, "q_out", (n, q_heads, dim), _BF16, device)
    rope_len = 0 if rope is None else rope.shape[0]
    table, n_seqs, max_pages = _table(page_table, device)
    rc = (_lib or load_library()).bd_kv_append(
        cache._ref, qp, q_heads, _arg(k, "k", kv_shape, _BF16, device), _arg(v, "v", kv_shape, _BF16, device), n,
        None if seq_ids is None else _arg(seq_ids, "seq_ids", (n,), _I32, device),
        _arg(positions, "positions", (n,), _I32, device), table, n_seqs, max_pages, None if rope is None else _arg(rope, "rope", (rope_len, dim), _F32, device), rope_len, qo,
        _raw_stream(stream, device))
    if rc:
        _check(rc, "bd_kv_append")


def bd_kv_read(cache: KVCache, page_table: torch.Tensor, offsets: torch.Tensor, k_out: torch.Tensor,
               v_out: torch.Tensor, stream=None) -> None:
    """The first offsets[i + 1] - offsets[i] cached tokens of sequence i, as bf16 rows offsets[i] .. of k_out and v_out."""
    device = cache.device
    table, n_seqs, max_pages = _table(page_table, device)
    shape = (k_out.shape[0], cache.kv_heads, cache.head_dim)
    rc = (_lib or load_library()).bd_kv_read(
        cache._ref, table, n_seqs, max_pages, _arg(offsets, "offsets", (n_seqs + 1,), _I32, device), shape[0],
        _arg(k_out, "k_out", shape, _BF16, device), _arg(v_out, "v_out", shape, _BF16, device), _raw_stream(stream, device))
    if rc:
        _check(rc, "bd_kv_read")


def bd_attention_workspace_size(cache: KVCache, n_seqs: int, q_heads: int) -> int:
    """Bytes of the workspace of bd_attention_decode (zero-filled once by the caller)."""
    return int(load_library().bd_attention_workspace_size(cache._ref, n_seqs, q_heads))


def bd_attention_decode(cache: KVCache, q: torch.Tensor, page_table: torch.Tensor, lengths: torch.Tensor,
                        out: torch.Tensor, workspace: torch.Tensor, scale: float | None = None, window: int = 0,
                        lse: torch.Tensor | None = None, stream=None) -> None:
    """Attention of one query per sequence, q [n_seqs, q_heads, head_dim], over its first lengths[i] cached tokens.

    `scale` defaults to head_dim ** -0.5; `window` > 0 lets a query see the last `window` tokens only.
    `workspace` is a zero-filled device buffer of at least bd_attention_workspace_size bytes (left
    ready for the next call)."""
    device = cache.device
    table, n_seqs, max_pages = _table(page_table, device)
    q_heads = q.shape[1] if q.dim() == 3 else 0
    shape = (n_seqs, q_heads, cache.head_dim)
    rc = (_lib or load_library()).bd_attention_decode(
        cache._ref, _arg(q, "q", shape, _BF16, device), q_heads, table, _arg(lengths, "lengths", (n_seqs,), _I32, device),
        n_seqs, max_pages, cache.head_dim ** -0.5 if scale is None else scale, max(-1, min(window, 0x7FFFFFFF)),
        _arg(out, "out", shape, _BF16, device),
        None if lse is None else _arg(lse, "lse", (n_seqs, q_heads), _F32, device),
        _arg(workspace, "workspace", workspace.shape, workspace.dtype, device), workspace.nbytes, _raw_stream(stream, device))
    if rc:
        _check(rc, "bd_attention_decode")


def bd_sample(logits: torch.Tensor, noise: torch.Tensor, ids: torch.Tensor, temperature: torch.Tensor | None = None,
              top_k: torch.Tensor | None = None, top_p: torch.Tensor | None = None, min_p: torch.Tensor | None = None,
              logprob: torch.Tensor | None = None, stream=None) -> None:
    """Draw ids [m] int32 from logits [m, vocab] (bf16 or fp32) with the given Gumbel noise, fp32 [m, vocab].

    `temperature`, `top_k` (int32), `top_p` and `min_p` hold one setting per row; None leaves the
    filter off (temperature 1).  `logprob` receives the drawn token's log probability before the filters."""
    half = logits.dtype is _BF16
    (lp, device), shape = _first(logits, "logits", _BF16 if half else _F32), logits.shape
    m, vocab = shape
    row = (m,)
    rc = (_lib or load_library()).bd_sample(
        lp, BD_LOGITS_BF16 if half else BD_LOGITS_F32, m, vocab,
        None if temperature is None else _arg(temperature, "temperature", row, _F32, device),
        None if top_k is None else _arg(top_k, "top_k", row, _I32, device),
        None if top_p is None else _arg(top_p, "top_p", row, _F32, device),
        None if min_p is None else _arg(min_p, "min_p", row, _F32, device), _arg(noise, "noise", shape, _F32, device),
        _arg(ids, "ids", row, _I32, device), None if logprob is None else _arg(logprob, "logprob", row, _F32, device),
        _raw_stream(stream, device))
    if rc:
        _check(rc, "bd_sample")
