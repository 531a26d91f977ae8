"""Sliding-window attention on GB300 (sm_103a): thin Python binding of libswa.so.

The functions here marshal torch tensors into the C ABI of ``include/swa.h``
(``swa_fwd``, ``swa_decode``, ``swa_cache_append``, ``swa_decode_append``,
``swa_prefill_chunk``, ``swa_paged_attend``, ``swa_paged_append``, the
``swa_pages_*`` calls and their workspace queries) and call it on the current
CUDA stream.  Every step of the computation runs in the library's
kernels; there is no fallback path.  If the library has not been built, the
first call raises (``build()`` compiles it in-tree with nvcc).

PyTorch is used for device memory and streams only.

Every call takes a ``stream``.  The paged calls (``swa_paged_*``, ``swa_pages_*``) make it the current
one while they run, so the results and workspaces that they allocate belong to it (a tensor that
another stream uses on needs ``record_stream``, as any does); the other calls allocate on
the current stream and launch on ``stream``.
"""
from __future__ import annotations

import ctypes
import os
import struct

from . import build as _build_mod

__all__ = [
    "SwaError", "build", "load_library", "library_path",
    "swa_fwd", "swa_decode", "swa_fwd_workspace_size", "swa_decode_workspace_size",
    "swa_check_device_error", "swa_status_string", "swa_abi_version",
    "SwaFwdParams", "SwaDecodeParams", "GLOBAL_FULL", "GLOBAL_SINK",
    "SwaCacheParams", "SwaChunkParams", "swa_cache_append", "swa_decode_append", "swa_prefill_chunk",
    "SwaDeviceErrors", "SwaDebugFaults", "swa_read_device_errors", "swa_debug_set_faults",
    "SwaPagedCache", "SwaPagedParams", "SwaPageTables", "SwaPagePool", "swa_paged_attend", "swa_paged_append",
    "swa_pages_reserve", "swa_pages_free", "swa_pages_fork", "swa_pages_compact", "swa_pages_copy",
]

_c_i64x3 = ctypes.c_int64 * 3
_c_i64x2 = ctypes.c_int64 * 2


class SwaFwdParams(ctypes.Structure):
    """Mirror of ``swa_fwd_params`` in include/swa.h."""

    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("q_strides", _c_i64x3), ("k_strides", _c_i64x3), ("v_strides", _c_i64x3),
        ("B", ctypes.c_int32), ("T", ctypes.c_int32), ("H_q", ctypes.c_int32), ("H_kv", ctypes.c_int32),
        ("d_h", ctypes.c_int32), ("window_left", ctypes.c_int32), ("window_right", ctypes.c_int32),
        ("scale", ctypes.c_float), ("global_idx", ctypes.c_void_p), ("n_global", ctypes.c_int32),
        ("o", ctypes.c_void_p), ("o_strides", _c_i64x3), ("lse", ctypes.c_void_p), ("row_counts", ctypes.c_void_p),
        ("global_mode", ctypes.c_int32), ("q_g", ctypes.c_void_p), ("k_g", ctypes.c_void_p), ("v_g", ctypes.c_void_p),
        ("qg_strides", _c_i64x3), ("kg_strides", _c_i64x3), ("vg_strides", _c_i64x3),
        ("dilation", ctypes.POINTER(ctypes.c_int32)),
    ]


class SwaDecodeParams(ctypes.Structure):
    """Mirror of ``swa_decode_params`` in include/swa.h."""

    _fields_ = [
        ("q", ctypes.c_void_p), ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
        ("slot_pos", ctypes.c_void_p), ("q_pos", ctypes.c_void_p),
        ("B", ctypes.c_int32), ("H_q", ctypes.c_int32), ("H_kv", ctypes.c_int32), ("d_h", ctypes.c_int32),
        ("W", ctypes.c_int32), ("scale", ctypes.c_float),
        ("o", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("row_counts", ctypes.c_void_p),
        ("window", ctypes.c_int32), ("n_sink", ctypes.c_int32),
    ]


class SwaCacheParams(ctypes.Structure):
    """Mirror of ``swa_cache_params`` in include/swa.h."""

    _fields_ = [
        ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p), ("slot_pos", ctypes.c_void_p),
        ("B", ctypes.c_int32), ("H_kv", ctypes.c_int32), ("d_h", ctypes.c_int32), ("n_slots", ctypes.c_int32),
        ("n_sink", ctypes.c_int32),
    ]


class SwaChunkParams(ctypes.Structure):
    """Mirror of ``swa_chunk_params`` in include/swa.h."""

    _fields_ = [
        ("q", ctypes.c_void_p), ("k_new", ctypes.c_void_p), ("v_new", ctypes.c_void_p), ("p0", ctypes.c_void_p),
        ("B", ctypes.c_int32), ("C", ctypes.c_int32), ("H_q", ctypes.c_int32), ("H_kv", ctypes.c_int32),
        ("d_h", ctypes.c_int32), ("window", ctypes.c_int32), ("scale", ctypes.c_float),
        ("o", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("row_counts", ctypes.c_void_p), ("append", ctypes.c_int32),
    ]


class SwaPagedCache(ctypes.Structure):
    """Mirror of ``swa_paged_cache`` in include/swa.h."""

    _fields_ = [
        ("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
        ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("H_kv", ctypes.c_int32), ("d_h", ctypes.c_int32),
        ("B", ctypes.c_int32), ("table_width", ctypes.c_int32),
    ]


class SwaPagedParams(ctypes.Structure):
    """Mirror of ``swa_paged_params`` in include/swa.h."""

    _fields_ = [
        ("q", ctypes.c_void_p), ("k_new", ctypes.c_void_p), ("v_new", ctypes.c_void_p), ("p0", ctypes.c_void_p),
        ("q_start", ctypes.c_void_p), ("q_strides", _c_i64x2), ("kn_strides", _c_i64x2), ("vn_strides", _c_i64x2),
        ("o_strides", _c_i64x2), ("N", ctypes.c_int32), ("H_q", ctypes.c_int32), ("max_q", ctypes.c_int32),
        ("window", ctypes.c_int32), ("n_sink", ctypes.c_int32), ("scale", ctypes.c_float), ("o", ctypes.c_void_p),
        ("lse", ctypes.c_void_p), ("row_counts", ctypes.c_void_p),
    ]


class SwaPageTables(ctypes.Structure):
    """Mirror of ``swa_page_tables`` in include/swa.h."""

    _fields_ = [
        ("table", ctypes.c_void_p), ("ref", ctypes.c_void_p), ("out_table", ctypes.c_void_p),
        ("out_ref", ctypes.c_void_p), ("B", ctypes.c_int32), ("width", ctypes.c_int32), ("n_pages", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
    ]


class SwaPagePool(ctypes.Structure):
    """Mirror of ``swa_page_pool`` in include/swa.h."""

    _fields_ = [
        ("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("layer_stride", ctypes.c_int64),
        ("n_layers", ctypes.c_int32), ("n_pages", ctypes.c_int32), ("H_kv", ctypes.c_int32),
        ("page_size", ctypes.c_int32), ("d_h", ctypes.c_int32),
    ]


class SwaDeviceErrors(ctypes.Structure):
    """Mirror of ``swa_device_errors`` in include/swa.h."""

    _fields_ = [("prefill", ctypes.c_uint32), ("split", ctypes.c_uint32), ("cache", ctypes.c_uint32)]


class SwaDebugFaults(ctypes.Structure):
    """Mirror of ``swa_debug_faults`` in include/swa.h."""

    _fields_ = [("band_stop_fill", ctypes.c_int32), ("split_stop_stage", ctypes.c_int32)]


# bits of the device error words
DEVERR_WAIT_TIMEOUT = 1
DEVERR_DRAIN_TIMEOUT = 2
DEVERR_GLOBAL_LIST = 4
DEVERR_BAD_POSITION = 1
DEVERR_CACHE_MISMATCH = 2
DEVERR_BAD_PAGE = 4
DEVERR_BOUNDS = 8
DEVERR_NO_PAGE = 16
DEVERR_BAD_REF = 32

GLOBAL_FULL = 0  # global tokens: full rows and columns
GLOBAL_SINK = 1  # attention sinks: key columns only, never right of a row's band

STATUS = {0: "SWA_OK", 1: "SWA_ERR_INVALID_ARG", 2: "SWA_ERR_UNSUPPORTED", 3: "SWA_ERR_CUDA",
          4: "SWA_ERR_TIMEOUT", 5: "SWA_ERR_WORKSPACE"}


class SwaError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        msg = f"{fn} returned {STATUS.get(status, status)}: {swa_status_string(status)}"
        if status == 3:
            msg += f" ({load_library().swa_last_error_string().decode()})"
        super().__init__(msg)


_lib = None


def library_path() -> str:
    return _build_mod.LIB


def build(force: bool = False, debug: bool = False) -> str:
    """Compile libswa.so for sm_103a (in-tree) and return its path; debug=True builds
    libswa_debug.so, whose kernels check every computed index (SWA_DEVERR_BOUNDS)."""
    return _build_mod.build(force=force, debug=debug)


def load_library(path: str | None = None):
    """Load libswa.so (raises if it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or library_path()
    if not os.path.exists(p):
        raise RuntimeError(f"libswa.so not found at {p}; call sliding_window_attention_swa_gb300.build() first")
    lib = ctypes.CDLL(p)
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    lib.swa_fwd_workspace_size.argtypes = [ctypes.POINTER(SwaFwdParams)]
    lib.swa_fwd_workspace_size.restype = sz
    lib.swa_fwd.argtypes = [ctypes.POINTER(SwaFwdParams), vp, sz, vp]
    lib.swa_fwd.restype = ctypes.c_int
    lib.swa_decode_workspace_size.argtypes = [ctypes.POINTER(SwaDecodeParams)]
    lib.swa_decode_workspace_size.restype = sz
    lib.swa_decode.argtypes = [ctypes.POINTER(SwaDecodeParams), vp, sz, vp]
    lib.swa_decode.restype = ctypes.c_int
    lib.swa_decode_noalloc.argtypes = [ctypes.POINTER(SwaDecodeParams), vp]
    lib.swa_decode_noalloc.restype = ctypes.c_int
    lib.swa_cache_append.argtypes = [ctypes.POINTER(SwaCacheParams), vp, vp, ctypes.c_int32, vp, vp]
    lib.swa_cache_append.restype = ctypes.c_int
    lib.swa_decode_append.argtypes = [ctypes.POINTER(SwaDecodeParams), vp, vp, vp, sz, vp]
    lib.swa_decode_append.restype = ctypes.c_int
    lib.swa_prefill_chunk_workspace_size.argtypes = [ctypes.POINTER(SwaChunkParams), ctypes.POINTER(SwaCacheParams)]
    lib.swa_prefill_chunk_workspace_size.restype = sz
    lib.swa_prefill_chunk.argtypes = [ctypes.POINTER(SwaChunkParams), ctypes.POINTER(SwaCacheParams), vp, sz, vp]
    lib.swa_prefill_chunk.restype = ctypes.c_int
    # (structures of the paged calls: a reference to one, or its packed bytes)
    lib.swa_paged_workspace_size.argtypes = [vp, vp]
    lib.swa_paged_workspace_size.restype = sz
    lib.swa_paged_attend.argtypes = [vp, vp, vp, sz, vp]
    lib.swa_paged_append.argtypes = [vp, vp, vp]
    lib.swa_pages_workspace_size.argtypes = [vp]
    lib.swa_pages_workspace_size.restype = sz
    lib.swa_pages_reserve.argtypes = [vp, vp, vp, vp, sz, vp]
    lib.swa_pages_free.argtypes = [vp, vp, ctypes.c_int32, vp]
    lib.swa_pages_fork.argtypes = [vp, vp, vp, vp, vp, sz, vp]
    lib.swa_pages_compact.argtypes = [vp, vp, vp, vp, sz, vp]
    lib.swa_pages_copy.argtypes = [vp, vp, vp, ctypes.c_int32, vp]
    for name in ("swa_paged_attend", "swa_paged_append", "swa_pages_reserve", "swa_pages_free", "swa_pages_fork",
                 "swa_pages_compact", "swa_pages_copy"):
        getattr(lib, name).restype = ctypes.c_int
    lib.swa_check_device_error.argtypes = [vp]
    lib.swa_check_device_error.restype = ctypes.c_int
    lib.swa_read_device_errors.argtypes = [vp, ctypes.POINTER(SwaDeviceErrors)]
    lib.swa_read_device_errors.restype = ctypes.c_int
    lib.swa_debug_set_faults.argtypes = [ctypes.POINTER(SwaDebugFaults)]
    lib.swa_debug_set_faults.restype = ctypes.c_int
    lib.swa_last_error_string.argtypes = []
    lib.swa_last_error_string.restype = ctypes.c_char_p
    lib.swa_status_string.argtypes = [ctypes.c_int]
    lib.swa_status_string.restype = ctypes.c_char_p
    lib.swa_abi_version.argtypes = []
    lib.swa_abi_version.restype = ctypes.c_int32
    if path is None:
        _lib = lib
    return lib


def use_library(lib):
    """Make `lib` (as returned by load_library(path)) the library the functions of this
    module call -- for example the debug build -- and return the previous one (None if
    none was loaded yet)."""
    global _lib
    prev, _lib = _lib, lib
    return prev


def swa_status_string(status: int) -> str:
    return load_library().swa_status_string(int(status)).decode()


def swa_abi_version() -> int:
    return int(load_library().swa_abi_version())


def _stream_handle(stream):
    import torch

    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check_bf16(name, t, ndim):
    import torch

    if t.dtype != torch.bfloat16 or not t.is_cuda or t.dim() != ndim or t.stride(-1) != 1:
        raise ValueError(f"{name}: expected a CUDA bf16 tensor of rank {ndim} with a contiguous last dim")


def fwd_params(q, k, v, window_left: int, window_right: int, scale: float, global_idx, o, lse, row_counts,
               global_mode: int = GLOBAL_FULL, qkv_g=None, dilation=None):
    """Fill a SwaFwdParams from tensors (q/k/v/o [B,T,H,d] bf16; lse/row_counts [B,H_q,T]).

    qkv_g: optional (q_g, k_g, v_g) separate global projections; dilation: optional
    per-query-head list of band dilations (host ints)."""
    B, T, Hq, D = q.shape
    p = SwaFwdParams()
    p.q, p.k, p.v, p.o = q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr()
    p.q_strides = _c_i64x3(*q.stride()[:3])
    p.k_strides = _c_i64x3(*k.stride()[:3])
    p.v_strides = _c_i64x3(*v.stride()[:3])
    p.o_strides = _c_i64x3(*o.stride()[:3])
    p.B, p.T, p.H_q, p.H_kv, p.d_h = B, T, Hq, k.shape[2], D
    p.window_left, p.window_right = int(window_left), int(window_right)
    p.scale = float(scale)
    p.global_idx = None if global_idx is None else global_idx.data_ptr()
    p.n_global = 0 if global_idx is None else int(global_idx.numel())
    p.lse = lse.data_ptr()
    p.row_counts = None if row_counts is None else row_counts.data_ptr()
    p.global_mode = int(global_mode)
    if qkv_g is not None:
        qg, kg, vg = qkv_g
        p.q_g, p.k_g, p.v_g = qg.data_ptr(), kg.data_ptr(), vg.data_ptr()
        p.qg_strides = _c_i64x3(*qg.stride()[:3])
        p.kg_strides = _c_i64x3(*kg.stride()[:3])
        p.vg_strides = _c_i64x3(*vg.stride()[:3])
    if dilation is not None:
        arr = (ctypes.c_int32 * Hq)(*[int(x) for x in dilation])
        p._dilation_keepalive = arr  # the C call reads it through the pointer
        p.dilation = ctypes.cast(arr, ctypes.POINTER(ctypes.c_int32))
    return p


def swa_fwd_workspace_size(params: SwaFwdParams) -> int:
    return int(load_library().swa_fwd_workspace_size(ctypes.byref(params)))


def swa_fwd(q, k, v, window_left: int, window_right: int, scale: float | None = None, global_idx=None, *,
            o=None, lse=None, row_counts=None, want_counts: bool = False, workspace=None, stream=None,
            global_mode: int = GLOBAL_FULL, q_g=None, k_g=None, v_g=None, dilation=None):
    """Banded attention over q [B,T,H_q,d], k/v [B,T,H_kv,d] (bf16, CUDA).

    Keys s with t - window_left <= s <= t + window_right (negative: unbounded side),
    plus global positions (int32 CUDA tensor, strictly increasing) used as
    global_mode says (GLOBAL_FULL rows and columns, GLOBAL_SINK pinned columns).
    q_g, k_g, v_g: separate global projections (shapes of q, k, v).  dilation:
    per-query-head band dilations (ints >= 1; window sides then count steps).
    Returns (o [B,T,H_q,d] bf16, lse [B,H_q,T] fp32, row_counts [B,H_q,T] int32 or None).
    """
    import torch

    lib = load_library()
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_bf16(name, t, 4)
    B, T, Hq, D = q.shape
    if scale is None:
        scale = D ** -0.5
    if global_idx is not None:
        if global_idx.dtype != torch.int32 or not global_idx.is_cuda:
            raise ValueError("global_idx: expected a CUDA int32 tensor")
        global_idx = global_idx.contiguous()
        if global_idx.numel() == 0:
            global_idx = None
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, Hq, T), dtype=torch.float32, device=q.device) if lse is None else lse
    if row_counts is None and want_counts:
        row_counts = torch.empty((B, Hq, T), dtype=torch.int32, device=q.device)
    qkv_g = None
    if q_g is not None or k_g is not None or v_g is not None:
        if q_g is None or k_g is None or v_g is None:
            raise ValueError("q_g, k_g and v_g go together")
        for name, t, ref in (("q_g", q_g, q), ("k_g", k_g, k), ("v_g", v_g, v)):
            _check_bf16(name, t, 4)
            if t.shape != ref.shape:
                raise ValueError(f"{name}: expected shape {tuple(ref.shape)}")
        qkv_g = (q_g, k_g, v_g)
    if dilation is not None and len(dilation) != Hq:
        raise ValueError(f"dilation: expected {Hq} entries")
    p = fwd_params(q, k, v, window_left, window_right, scale, global_idx, o, lse, row_counts, global_mode, qkv_g,
                   dilation)
    need = int(lib.swa_fwd_workspace_size(ctypes.byref(p)))
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = _ptr(workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.swa_fwd(ctypes.byref(p), ws_ptr, ws_bytes, _stream_handle(stream))
    if st != 0:
        raise SwaError("swa_fwd", st)
    return o, lse, row_counts


def decode_params(q, k_cache, v_cache, slot_pos, q_pos, scale: float, o, lse, row_counts, window: int = 0,
                  n_sink: int = 0):
    B, Hq, D = q.shape
    p = SwaDecodeParams()
    p.q, p.k_cache, p.v_cache = q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr()
    p.slot_pos, p.q_pos = slot_pos.data_ptr(), q_pos.data_ptr()
    p.B, p.H_q, p.H_kv, p.d_h, p.W = B, Hq, k_cache.shape[1], D, k_cache.shape[2]
    p.scale = float(scale)
    p.o, p.lse = o.data_ptr(), lse.data_ptr()
    p.row_counts = None if row_counts is None else row_counts.data_ptr()
    p.window, p.n_sink = int(window), int(n_sink)
    return p


def swa_decode_workspace_size(params: SwaDecodeParams) -> int:
    return int(load_library().swa_decode_workspace_size(ctypes.byref(params)))


def swa_decode(q, k_cache, v_cache, slot_pos, q_pos, scale: float | None = None, *, o=None, lse=None,
               row_counts=None, want_counts: bool = False, workspace=None, stream=None, window: int = 0,
               n_sink: int = 0):
    """Ring-buffer decode: q [B,H_q,d], caches [B,H_kv,W,d] (bf16), slot_pos [B,W], q_pos [B] (int32).

    window: the window in positions (0: the number of slots W); n_sink: the first
    positions that are always attended.  Returns (o [B,H_q,d] bf16, lse [B,H_q] fp32,
    row_counts [B,H_q] int32 or None).
    """
    import torch

    lib = load_library()
    _check_bf16("q", q, 3)
    _check_bf16("k_cache", k_cache, 4)
    _check_bf16("v_cache", v_cache, 4)
    for name, t in (("q", q), ("k_cache", k_cache), ("v_cache", v_cache), ("slot_pos", slot_pos), ("q_pos", q_pos)):
        if not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous tensor")
    if slot_pos.dtype != torch.int32 or q_pos.dtype != torch.int32:
        raise ValueError("slot_pos and q_pos must be int32")
    B, Hq, D = q.shape
    if scale is None:
        scale = D ** -0.5
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device) if lse is None else lse
    if row_counts is None and want_counts:
        row_counts = torch.empty((B, Hq), dtype=torch.int32, device=q.device)
    p = decode_params(q, k_cache, v_cache, slot_pos, q_pos, scale, o, lse, row_counts, window, n_sink)
    need = int(lib.swa_decode_workspace_size(ctypes.byref(p)))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    st = lib.swa_decode(ctypes.byref(p), _ptr(workspace), ws_bytes, _stream_handle(stream))
    if st != 0:
        raise SwaError("swa_decode", st)
    return o, lse, row_counts


def cache_params(k_cache, v_cache, slot_pos, n_sink: int = 0) -> SwaCacheParams:
    """caches bf16 [B,H_kv,n_slots,d] and slot_pos int32 [B,n_slots] (contiguous, CUDA)."""
    c = SwaCacheParams()
    c.k_cache, c.v_cache, c.slot_pos = k_cache.data_ptr(), v_cache.data_ptr(), slot_pos.data_ptr()
    c.B, c.H_kv, c.n_slots, c.d_h = k_cache.shape
    c.n_sink = int(n_sink)
    return c


def _check_cache(k_cache, v_cache, slot_pos):
    import torch

    _check_bf16("k_cache", k_cache, 4)
    _check_bf16("v_cache", v_cache, 4)
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache), ("slot_pos", slot_pos)):
        if not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous tensor")
    if slot_pos.dtype != torch.int32 or v_cache.shape != k_cache.shape or tuple(slot_pos.shape) != tuple(k_cache.shape[::2]):
        raise ValueError("slot_pos: expected int32 [B, n_slots] matching the caches")


def swa_cache_append(k_cache, v_cache, slot_pos, k_new, v_new, p0, *, n_sink: int = 0, stream=None) -> None:
    """Append k_new/v_new [B,n,H_kv,d] (positions p0[b] + i, p0 int32 CUDA [B]) to the
    ring cache in place (slot rule of include/swa.h with n_sink pinned sinks)."""
    import torch

    _check_cache(k_cache, v_cache, slot_pos)
    for name, t in (("k_new", k_new), ("v_new", v_new)):
        _check_bf16(name, t, 4)
        if not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous tensor")
    if p0.dtype != torch.int32 or not p0.is_contiguous():
        raise ValueError("p0: expected a contiguous int32 tensor")
    c = cache_params(k_cache, v_cache, slot_pos, n_sink)
    st = load_library().swa_cache_append(ctypes.byref(c), _ptr(k_new), _ptr(v_new), int(k_new.shape[1]), _ptr(p0),
                                         _stream_handle(stream))
    if st != 0:
        raise SwaError("swa_cache_append", st)


def swa_decode_append(q, k_cache, v_cache, slot_pos, q_pos, k_new, v_new, scale: float | None = None, *, o=None,
                      lse=None, want_counts: bool = False, workspace=None, stream=None, window: int = 0,
                      n_sink: int = 0):
    """swa_decode with the current token's k_new/v_new [B,H_kv,d] appended to the cache
    (in place) in the same pass.  Returns (o, lse, row_counts or None)."""
    import torch

    lib = load_library()
    _check_bf16("q", q, 3)
    _check_cache(k_cache, v_cache, slot_pos)
    for name, t in (("k_new", k_new), ("v_new", v_new)):
        _check_bf16(name, t, 3)
        if not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous tensor")
    B, Hq, D = q.shape
    if scale is None:
        scale = D ** -0.5
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device) if lse is None else lse
    row_counts = torch.empty((B, Hq), dtype=torch.int32, device=q.device) if want_counts else None
    p = decode_params(q, k_cache, v_cache, slot_pos, q_pos, scale, o, lse, row_counts, window, n_sink)
    need = int(lib.swa_decode_workspace_size(ctypes.byref(p)))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    st = lib.swa_decode_append(ctypes.byref(p), _ptr(k_new), _ptr(v_new), _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _stream_handle(stream))
    if st != 0:
        raise SwaError("swa_decode_append", st)
    return o, lse, row_counts


def chunk_params(q, k_new, v_new, p0, window: int, scale: float, o, lse, row_counts, append: bool) -> SwaChunkParams:
    B, C, Hq, D = q.shape
    p = SwaChunkParams()
    p.q, p.k_new, p.v_new, p.p0 = q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), p0.data_ptr()
    p.B, p.C, p.H_q, p.H_kv, p.d_h = B, C, Hq, k_new.shape[2], D
    p.window, p.scale = int(window), float(scale)
    p.o, p.lse = o.data_ptr(), lse.data_ptr()
    p.row_counts = None if row_counts is None else row_counts.data_ptr()
    p.append = 1 if append else 0
    return p


def swa_prefill_chunk(q, k_new, v_new, k_cache, v_cache, slot_pos, p0, window: int, scale: float | None = None, *,
                      append: bool = False, o=None, lse=None, want_counts: bool = False, workspace=None,
                      stream=None, n_sink: int = 0):
    """Chunked prefill: q [B,C,H_q,d] and the chunk's k_new/v_new [B,C,H_kv,d] at positions
    p0[b] + i attend to the ring cache's history and to the chunk (causal window), and to
    the cache's n_sink pinned sinks.  append: afterwards the chunk joins the cache.  Returns (o [B,C,H_q,d], lse [B,H_q,C],
    row_counts or None)."""
    import torch

    lib = load_library()
    for name, t in (("q", q), ("k_new", k_new), ("v_new", v_new)):
        _check_bf16(name, t, 4)
        if not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous tensor")
    _check_cache(k_cache, v_cache, slot_pos)
    if p0.dtype != torch.int32 or not p0.is_contiguous():
        raise ValueError("p0: expected a contiguous int32 tensor")
    B, C, Hq, D = q.shape
    if scale is None:
        scale = D ** -0.5
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, Hq, C), dtype=torch.float32, device=q.device) if lse is None else lse
    row_counts = torch.empty((B, Hq, C), dtype=torch.int32, device=q.device) if want_counts else None
    p = chunk_params(q, k_new, v_new, p0, window, scale, o, lse, row_counts, append)
    c = cache_params(k_cache, v_cache, slot_pos, n_sink)
    need = int(lib.swa_prefill_chunk_workspace_size(ctypes.byref(p), ctypes.byref(c)))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    st = lib.swa_prefill_chunk(ctypes.byref(p), ctypes.byref(c), _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _stream_handle(stream))
    if st != 0:
        raise SwaError("swa_prefill_chunk", st)
    return o, lse, row_counts


# The paged calls are made once a layer and step, so what they cost on the host counts: arguments
# are packed in one go (the layouts of the structures above, without trailing padding), and
# checks look at a tensor's device index, not at device objects.
_paged_ws_size: dict = {}
_PAGED_PARAMS = struct.Struct("5P8q5if3P")
_PAGED_CACHE = struct.Struct("3P6i")
_PAGE_TABLES = struct.Struct("4P4i")
_PAGE_POOL = struct.Struct("2Pq5i")


def _packed(layout, *values) -> bytes:
    try:
        return layout.pack(*values)
    except struct.error as e:
        raise ValueError(f"a size, window or hint that 32 bits do not hold: {e}") from None


def _int32(name, value) -> int:
    """An argument of its own (ctypes would pass its low 32 bits)."""
    value = int(value)
    if not -(1 << 31) <= value < 1 << 31:
        raise ValueError(f"{name}: {value} does not fit 32 bits")
    return value


def _i32_wrong(name, shape, index):
    return ValueError(f"{name}: expected a contiguous int32 tensor of shape {list(shape)} on cuda:{index}")


def _device_index(name, t) -> int:
    """The library's calls go to the current device: tensors of another one are refused."""
    import torch

    index = t.get_device()
    if index < 0 or index != torch._C._cuda_getDevice():
        raise ValueError(f"{name}: expected a tensor on the current CUDA device, got {t.device}")
    return index


def _own_workspace(workspace, index: int) -> None:
    """A workspace that the caller gives: the kernels write to its address, whatever device that is on."""
    if workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError(f"workspace: expected a contiguous tensor on cuda:{index}")


def _raw_stream(index: int) -> int:
    import torch

    return torch._C._cuda_getCurrentRawStream(index)


def _on(stream, call, *args, **kw):
    """The call with `stream` as the current one, so that the memory that it allocates, and lets go
    of when it returns, belongs to that stream."""
    import torch

    with torch.cuda.stream(stream):
        return call(*args, **kw)


def _paged_cache(k_pages, v_pages, page_table, p0, q_start, N: int):
    """(device index, swa_paged_cache, H_kv, d_h), the cache and the batch's lists checked."""
    import torch

    index = _device_index("k_pages", k_pages)
    shape, bf16, i32 = k_pages.shape, torch.bfloat16, torch.int32
    for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
        if t.dtype is not bf16 or t.get_device() != index or len(shape) != 4 or t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous CUDA bf16 tensor [n_pages, H_kv, page_size, d], the same "
                             "for keys and values")
    if page_table.dim() != 2 or page_table.dtype is not i32 or page_table.get_device() != index or \
            not page_table.is_contiguous():
        raise _i32_wrong("page_table", ("B", "table_width"), index)
    B, width = page_table.shape
    if p0.dtype is not i32 or p0.get_device() != index or p0.shape != (B,) or not p0.is_contiguous():
        raise _i32_wrong("p0", (B,), index)
    if q_start is None:
        if N != B:
            raise ValueError(f"q_start: needed unless every sequence has one token ({N} rows, {B} sequences)")
    elif q_start.dtype is not i32 or q_start.get_device() != index or q_start.shape != (B + 1,) or \
            not q_start.is_contiguous():
        raise _i32_wrong("q_start", (B + 1,), index)
    n_pages, H_kv, page_size, D = shape
    return index, _packed(_PAGED_CACHE, k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), n_pages,
                          page_size, H_kv, D, B, width), H_kv, D


def _rows(name, t, index: int, shape) -> tuple:
    """The token and head strides of packed rows [N, heads, d], checked."""
    import torch

    st = t.stride()
    if t.dtype is not torch.bfloat16 or t.get_device() != index or t.shape != shape or st[2] != 1:
        raise ValueError(f"{name}: expected a bf16 tensor {list(shape)} with a contiguous last dim on cuda:{index}")
    return st[0], st[1]


def _new_rows(k_new, v_new, index: int, shape) -> tuple:
    """(addresses, strides) of the new tokens' keys and values (zeros without them)."""
    if k_new is None and v_new is None:
        return (0, 0), (0, 0, 0, 0)
    if k_new is None or v_new is None:
        raise ValueError("k_new and v_new go together")
    st = _rows("k_new", k_new, index, shape) + _rows("v_new", v_new, index, shape)
    return (k_new.data_ptr(), v_new.data_ptr()), st


def swa_paged_attend(q, k_pages, v_pages, page_table, p0, window: int = 0, scale: float | None = None, *, q_start=None,
                     n_sink: int = 0, max_q: int = 0, k_new=None, v_new=None, o=None, lse=None, row_counts=None,
                     want_counts: bool = False, workspace=None, stream=None):
    """Attention of new tokens over a paged cache: q [N,H_q,d] (bf16, any token and head strides),
    pools [n_pages,H_kv,page_size,d], page_table int32 [B,table_width], p0 int32 [B].

    Rows q_start[b] .. q_start[b+1]-1 (int32 [B+1]; None: one row a sequence) are sequence b's
    new tokens at positions p0[b] + i; the query at position t keeps the keys at positions s <= t
    with s > t - window (window 0: all) or s < n_sink.  k_new, v_new [N,H_kv,d]: stored in their
    pages first.  max_q: the most new tokens of one sequence if known (a hint; without it a
    batch with q_start goes to the kernel for many rows, which mostly takes 6 to 14% longer for
    one token a sequence).  Rows outside every sequence keep what o, lse and row_counts hold.
    Returns (o [N,H_q,d] bf16, lse [N,H_q] fp32, row_counts [N,H_q] int32 or None).
    """
    import torch

    if stream is not None:
        return _on(stream, swa_paged_attend, q, k_pages, v_pages, page_table, p0, window, scale, q_start=q_start,
                   n_sink=n_sink, max_q=max_q, k_new=k_new, v_new=v_new, o=o, lse=lse, row_counts=row_counts,
                   want_counts=want_counts, workspace=workspace)
    lib = load_library()
    if q.dim() != 3:
        raise ValueError("q: expected [N, H_q, d]")
    N, Hq, D = shape = q.shape
    index, cache, H_kv, d_h = _paged_cache(k_pages, v_pages, page_table, p0, q_start, N)
    q_st = _rows("q", q, index, (N, Hq, d_h))
    new, new_st = _new_rows(k_new, v_new, index, (N, H_kv, d_h))
    device = q.device
    if o is None:
        o, o_st = torch.empty(shape, dtype=torch.bfloat16, device=device), (Hq * D, D)
    else:
        o_st = _rows("o", o, index, shape)
    if lse is None:
        lse = torch.empty((N, Hq), dtype=torch.float32, device=device)
    elif lse.dtype is not torch.float32 or lse.get_device() != index or lse.shape != (N, Hq) or not lse.is_contiguous():
        raise ValueError(f"lse: expected a contiguous fp32 tensor {[N, Hq]} on cuda:{index}")
    if row_counts is None:
        if want_counts:
            row_counts = torch.empty((N, Hq), dtype=torch.int32, device=device)
    elif row_counts.dtype is not torch.int32 or row_counts.get_device() != index or row_counts.shape != (N, Hq) or \
            not row_counts.is_contiguous():
        raise _i32_wrong("row_counts", (N, Hq), index)
    if N == 0:
        return o, lse, row_counts
    params = _packed(
        _PAGED_PARAMS, q.data_ptr(), *new, p0.data_ptr(), 0 if q_start is None else q_start.data_ptr(), *q_st,
        *new_st, *o_st, N, Hq, int(max_q), int(window), int(n_sink), D ** -0.5 if scale is None else float(scale),
        o.data_ptr(), lse.data_ptr(), 0 if row_counts is None else row_counts.data_ptr())
    if workspace is None:
        # (asked once for each of what it depends on: the question takes 2 us of a 24 us call; more than
        # 16 tokens a sequence are many rows for every group, so a longer chunk is no other key)
        key = lib._name, index, Hq, H_kv, d_h, min(max_q, 17), q_start is None
        size = _paged_ws_size.get(key)
        if size is None:
            size = lib.swa_paged_workspace_size(params, cache)
            if size:  # (0: refused, below)
                _paged_ws_size[key] = size
        workspace = torch.empty(size or 1, dtype=torch.uint8, device=device)
    else:
        _own_workspace(workspace, index)
    st = lib.swa_paged_attend(params, cache, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                              _raw_stream(index))
    if st != 0:
        raise SwaError("swa_paged_attend", st)
    return o, lse, row_counts


def swa_paged_append(k_pages, v_pages, page_table, k_new, v_new, p0, *, q_start=None, stream=None) -> None:
    """Store k_new/v_new [N,H_kv,d] (packed rows as in swa_paged_attend) in their pages."""
    if stream is not None:
        return _on(stream, swa_paged_append, k_pages, v_pages, page_table, k_new, v_new, p0, q_start=q_start)
    N = k_new.shape[0]
    index, cache, H_kv, D = _paged_cache(k_pages, v_pages, page_table, p0, q_start, N)
    new, new_st = _new_rows(k_new, v_new, index, (N, H_kv, D))
    if N == 0:
        return
    params = _packed(_PAGED_PARAMS, 0, *new, p0.data_ptr(), 0 if q_start is None else q_start.data_ptr(), 0, 0,
                     *new_st, 0, 0, N, 0, 0, 0, 0, 0.0, 0, 0, 0)
    st = load_library().swa_paged_append(params, cache, _raw_stream(index))
    if st != 0:
        raise SwaError("swa_paged_append", st)


def _lists(index: int, *named) -> None:
    """Each (name, tensor, shape): a contiguous int32 tensor of that shape on the device."""
    import torch

    for name, t, shape in named:
        if t.dtype is not torch.int32 or t.get_device() != index or t.shape != shape or not t.is_contiguous():
            raise _i32_wrong(name, shape, index)


def _page_tables(page_table, ref, page_size: int, out_table, out_ref):
    """(device index, swa_page_tables, B), checked."""
    index = _device_index("page_table", page_table)
    if page_table.dim() != 2 or ref.dim() != 1:
        raise ValueError("page_table: expected int32 [B, width], and ref int32 [n_pages]")
    shape, n = page_table.shape, ref.shape
    _lists(index, ("page_table", page_table, shape), ("ref", ref, n), ("out_table", out_table, shape),
           ("out_ref", out_ref, n))
    return index, _packed(_PAGE_TABLES, page_table.data_ptr(), ref.data_ptr(), out_table.data_ptr(),
                          out_ref.data_ptr(), shape[0], shape[1], n[0], int(page_size)), shape[0]


def _page_pool(k_pages, v_pages):
    """(device index, swa_page_pool, page_size) of a pool [n_pages,H_kv,page_size,d] or
    [n_layers,n_pages,H_kv,page_size,d] whose layers are each contiguous."""
    import torch

    index = _device_index("k_pages", k_pages)
    shape, st = k_pages.shape, k_pages.stride()
    layers = shape[0] if len(shape) == 5 else 1
    if len(shape) not in (4, 5) or v_pages.shape != shape or v_pages.stride() != st or \
            k_pages.dtype is not torch.bfloat16 or v_pages.dtype is not torch.bfloat16 or v_pages.get_device() != index:
        raise ValueError("k_pages, v_pages: expected bf16 [n_pages, H_kv, page_size, d] or [n_layers, n_pages, H_kv, "
                         f"page_size, d], the same shape and strides for both, on cuda:{index}")
    n, H, ps, D = shape[-4:]
    if st[-4:] != (H * ps * D, ps * D, D, 1) and not (k_pages if len(shape) == 4 else k_pages[0]).is_contiguous():
        raise ValueError("k_pages, v_pages: expected each layer's pages to be contiguous")
    return index, _packed(_PAGE_POOL, k_pages.data_ptr(), v_pages.data_ptr(), st[0] if len(shape) == 5 else 0, layers,
                          n, H, ps, D), ps


def _pages_workspace(lib, tables, workspace, device):
    import torch

    if workspace is None:
        workspace = torch.empty(lib.swa_pages_workspace_size(tables) or 1, dtype=torch.uint8, device=device)
    else:
        _own_workspace(workspace, device.index)
    return workspace, workspace.numel() * workspace.element_size()


def swa_pages_reserve(page_table, ref, first, end, page_size: int, *, workspace=None, stream=None) -> None:
    """Give row b of page_table (in place, with ref) a page for every position in [first[b], end[b])
    that has none: the lowest free pages, in the order of rows and entries."""
    if stream is not None:
        return _on(stream, swa_pages_reserve, page_table, ref, first, end, page_size, workspace=workspace)
    lib = load_library()
    index, t, B = _page_tables(page_table, ref, page_size, page_table, ref)
    _lists(index, ("first", first, (B,)), ("end", end, (B,)))
    workspace, n = _pages_workspace(lib, t, workspace, page_table.device)
    st = lib.swa_pages_reserve(t, first.data_ptr(), end.data_ptr(), workspace.data_ptr(), n, _raw_stream(index))
    if st != 0:
        raise SwaError("swa_pages_reserve", st)


def swa_pages_free(page_table, ref, below, page_size: int, *, n_sink: int = 0, out_table=None, out_ref=None,
                   stream=None):
    """Row b gives up its pages whose positions all lie below below[b] and past the first n_sink
    positions' pages (below[b] < 0: all its pages).  In place unless out_table and out_ref are
    given.  Returns (out_table, out_ref)."""
    if stream is not None:
        return _on(stream, swa_pages_free, page_table, ref, below, page_size, n_sink=n_sink, out_table=out_table,
                   out_ref=out_ref)
    out_table, out_ref = page_table if out_table is None else out_table, ref if out_ref is None else out_ref
    index, t, B = _page_tables(page_table, ref, page_size, out_table, out_ref)
    _lists(index, ("below", below, (B,)))
    st = load_library().swa_pages_free(t, below.data_ptr(), _int32("n_sink", n_sink), _raw_stream(index))
    if st != 0:
        raise SwaError("swa_pages_free", st)
    return out_table, out_ref


def swa_pages_fork(k_pages, v_pages, page_table, ref, src, seq_len, *, out_table=None, out_ref=None, workspace=None,
                   stream=None):
    """New row i continues row src[i] (-1: empty) of page_table, which holds seq_len[src[i]] tokens:
    full pages are shared, a last page that is not full stays with the first row whose last page it
    is (with none if it is a full page of some row) and is copied for each other one (in every
    layer of k_pages/v_pages [n_layers,][n_pages,H_kv,page_size,d]).  out_table (not page_table
    itself; new if not given) and out_ref (in place if not given) are written whole.  Returns
    (out_table, out_ref)."""
    import torch

    if stream is not None:
        return _on(stream, swa_pages_fork, k_pages, v_pages, page_table, ref, src, seq_len, out_table=out_table,
                   out_ref=out_ref, workspace=workspace)
    lib = load_library()
    pool_index, pool, page_size = _page_pool(k_pages, v_pages)
    out_table = torch.empty_like(page_table) if out_table is None else out_table
    out_ref = ref if out_ref is None else out_ref
    index, t, B = _page_tables(page_table, ref, page_size, out_table, out_ref)
    _lists(index, ("src", src, (B,)), ("seq_len", seq_len, (B,)))
    workspace, n = _pages_workspace(lib, t, workspace, page_table.device)
    st = lib.swa_pages_fork(t, pool, src.data_ptr(), seq_len.data_ptr(), workspace.data_ptr(), n,
                            _raw_stream(pool_index))
    if st != 0:
        raise SwaError("swa_pages_fork", st)
    return out_table, out_ref


def swa_pages_compact(k_pages, v_pages, page_table, ref, *, out_table=None, out_ref=None, n_live=None, workspace=None,
                      stream=None):
    """Move the pool's live pages (ref > 0) to its low end, in every layer, and change page_table and
    ref accordingly (in place unless out_table and out_ref are given).  Returns (out_table,
    out_ref, n_live int32 [1], on the device)."""
    import torch

    if stream is not None:
        return _on(stream, swa_pages_compact, k_pages, v_pages, page_table, ref, out_table=out_table, out_ref=out_ref,
                   n_live=n_live, workspace=workspace)
    lib = load_library()
    pool_index, pool, page_size = _page_pool(k_pages, v_pages)
    out_table, out_ref = page_table if out_table is None else out_table, ref if out_ref is None else out_ref
    index, t, _ = _page_tables(page_table, ref, page_size, out_table, out_ref)
    n_live = torch.empty(1, dtype=torch.int32, device=page_table.device) if n_live is None else n_live
    _lists(index, ("n_live", n_live, (1,)))
    workspace, n = _pages_workspace(lib, t, workspace, page_table.device)
    st = lib.swa_pages_compact(t, pool, n_live.data_ptr(), workspace.data_ptr(), n, _raw_stream(pool_index))
    if st != 0:
        raise SwaError("swa_pages_compact", st)
    return out_table, out_ref, n_live


def swa_pages_copy(k_pages, v_pages, src, dst, *, stream=None) -> None:
    """Copy page src[i] to page dst[i] in every layer (int32 lists; the dst distinct, none also a src)."""
    if stream is not None:
        return _on(stream, swa_pages_copy, k_pages, v_pages, src, dst)
    index, pool, _ = _page_pool(k_pages, v_pages)
    if src.dim() != 1:
        raise ValueError("src: expected int32 [n]")
    _lists(index, ("src", src, src.shape), ("dst", dst, src.shape))
    st = load_library().swa_pages_copy(pool, src.data_ptr(), dst.data_ptr(), _int32("n", src.shape[0]), _raw_stream(index))
    if st != 0:
        raise SwaError("swa_pages_copy", st)


def swa_check_device_error(stream=None) -> None:
    """Synchronise the stream and raise if a kernel gave up on a bounded wait or found
    device data breaking its contract."""
    st = load_library().swa_check_device_error(_stream_handle(stream))
    if st != 0:
        raise SwaError("swa_check_device_error", st)


def swa_read_device_errors(stream=None) -> tuple[int, dict]:
    """Synchronise the stream, read and clear the device error words: (status, words)
    with words = {"prefill": bits, "split": bits, "cache": bits}."""
    e = SwaDeviceErrors()
    st = load_library().swa_read_device_errors(_stream_handle(stream), ctypes.byref(e))
    return int(st), {"prefill": int(e.prefill), "split": int(e.split), "cache": int(e.cache)}


def swa_debug_set_faults(band_stop_fill: int = -1, split_stop_stage: int = -1) -> None:
    """Failure-detection test hook (process-wide): the prefill kernel's producer stops
    before ring fill band_stop_fill, the split pass's before stage split_stop_stage
    (-1: off).  Called with no arguments it restores normal operation."""
    f = SwaDebugFaults(int(band_stop_fill), int(split_stop_stage))
    st = load_library().swa_debug_set_faults(ctypes.byref(f))
    if st != 0:
        raise SwaError("swa_debug_set_faults", st)
