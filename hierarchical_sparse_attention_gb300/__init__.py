"""Python binding of libhs, the HiSparse decode-step resolver / swap-in for GB300.

Argument marshalling only: every call goes straight to the C ABI declared in
``include/hs.h`` (same names), and every step of the path runs in the library's CUDA
kernels. Arguments that are device arrays accept a torch CUDA tensor (its
``data_ptr()``) or a raw address; host pools accept a numpy array or a raw address;
``stream`` accepts a ``torch.cuda.Stream``, a raw ``cudaStream_t`` or None (the legacy
default stream). A non-OK status raises :class:`HsError` carrying the status code. The 4-bit
cache's calls and the batches' (``hs_fp4_*``, ``hs_pages_*``, ``hs_batch_plan``, ``hs_fp8_*``,
``hs_chunk_mla``) also refuse, with ValueError, a tensor that is not on
the current CUDA device, a page pool whose tensors are not, and a tensor whose elements are of another
type than the call's (bf16 arrays may be given as their 16-bit patterns).

The in-tree ``libhs.so`` is loaded on first use; every entry point raises ImportError
if it has not been built (``python -m hierarchical_sparse_attention_gb300.build``).
There is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhs.so")

HS_OK, HS_ERR_INVALID_ARG, HS_ERR_INVALID_CONFIG, HS_ERR_CUDA, HS_ERR_DEVICE_FLAGGED, HS_ERR_TIMEOUT = range(6)
HS_FLAG_TOKEN, HS_FLAG_DUP, HS_FLAG_STATE, HS_FLAG_HOSTROW, HS_FLAG_DEVROW, HS_FLAG_SEQLEN = 1, 2, 4, 8, 16, 32
HS_FLAG_ORDER = 64
HS_FLAG_TIMEOUT = 128
HS_FLAG_NOPAGE = 256
HS_FLAG_FULL = 512
HS_MAX_MLA_SPLITS = 16
HS_MAX_TOP_K, HS_MAX_HOT_SLOTS, HS_MAX_LAYERS = 4096, 16384, 8

# Every symbol include/hs.h declares (checked against the library by the tests).
EXPORTS = ("hs_workspace_bytes", "hs_create", "hs_resolve", "hs_backup", "hs_get_error", "hs_destroy",
           "hs_status_str", "hs_host_register", "hs_host_unregister", "hs_resolve_noalloc",
           "hs_invalidate_tokens", "hs_invalidate_host_rows", "hs_resolve_layers", "hs_gather",
           "hs_resolve_spec", "hs_backup_spec", "hs_reset_hints", "hs_sparse_mla_workspace_bytes",
           "hs_sparse_mla_decode", "hs_launch_shape", "hs_resolve_spec_layers", "hs_gather_spec",
           "hs_host_numa_node", "hs_host_bind_node", "hs_sparse_mla_launches",
           "hs_fp4_pack_rows", "hs_fp4_unpack_rows", "hs_fp4_mla_splits", "hs_fp4_mla_workspace_bytes",
           "hs_fp4_sparse_mla_decode", "hs_fp4_window_mla_decode", "hs_pages_workspace_bytes", "hs_pages_init",
           "hs_pages_extend", "hs_pages_fork", "hs_pages_free", "hs_pages_compact", "hs_batch_plan",
           "hs_fp8_pack_rows", "hs_fp8_unpack_rows", "hs_chunk_mla_workspace_bytes", "hs_chunk_mla")
HS_MAX_SPEC_QUERIES = 8
HS_NOALLOC_MAX_LAYERS = 8
HS_FP4_ROW_BYTES = 416
HS_MAX_FP4_MLA_REQUESTS = 1 << 20
HS_MAX_PAGE_REQUESTS = 65536
HS_MAX_PAGE_ENTRIES = 1 << 20
HS_FP8_ROW_BYTES = 656
HS_MAX_BATCH_ENTRIES = 65536
HS_MAX_BATCH_TOKENS = 1 << 20


class hs_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("max_requests", "top_k", "hot_slots", "row_bytes", "num_layers",
                                              "page_size", "max_context", "max_pages", "host_row_stride")]


class hs_page_pool(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("num_requests", "max_pages", "num_pages", "page_size", "row_bytes",
                                               "num_layers")] +
                [("device_pools", ctypes.c_void_p * HS_MAX_LAYERS)] +
                [(n, ctypes.c_void_p) for n in ("resident_pages", "page_refs", "free_pages", "free_count",
                                                "error_flags", "workspace")] +
                [("workspace_bytes", ctypes.c_size_t)])
    device = None  # the CUDA device of the tensors it was made of; None: raw addresses only


class HsError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {hs_status_str(status)} (status {status})")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m hierarchical_sparse_attention_gb300.build` (nvcc, sm_103a)")
    lib = ctypes.CDLL(LIB_PATH)
    P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    cfgp = ctypes.POINTER(hs_config)
    lib.hs_workspace_bytes.argtypes = [cfgp]
    lib.hs_workspace_bytes.restype = sz
    lib.hs_create.argtypes = [cfgp, P, P, i64, i64, P, ctypes.POINTER(P)]
    lib.hs_create.restype = ctypes.c_int
    lib.hs_resolve.argtypes = [P, i32] + [P] * 10 + [P]
    lib.hs_resolve.restype = ctypes.c_int
    lib.hs_backup.argtypes = [P, i32, P, P, P, P, P]
    lib.hs_backup.restype = ctypes.c_int
    lib.hs_resolve_layers.argtypes = [P, i32] + [P] * 10 + [i32, P]
    lib.hs_resolve_layers.restype = ctypes.c_int
    lib.hs_gather.argtypes = [P, i32, P, i32, i32, P]
    lib.hs_sparse_mla_workspace_bytes.argtypes = [i32, i32, i32]
    lib.hs_sparse_mla_workspace_bytes.restype = sz
    lib.hs_sparse_mla_launches.argtypes = [i32, i32, i32]
    lib.hs_sparse_mla_launches.restype = i32
    lib.hs_sparse_mla_decode.argtypes = [i32, i32, i32, i32, P, P, i64, P, ctypes.c_float, P, P, P, sz, P, P]
    lib.hs_sparse_mla_decode.restype = ctypes.c_int
    lib.hs_reset_hints.argtypes = [P, P]
    lib.hs_reset_hints.restype = ctypes.c_int
    lib.hs_launch_shape.argtypes = [P, ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32)]
    lib.hs_launch_shape.restype = ctypes.c_int
    lib.hs_resolve_spec.argtypes = [P, i32, i32] + [P] * 10 + [P]
    lib.hs_resolve_spec.restype = ctypes.c_int
    lib.hs_resolve_spec_layers.argtypes = [P, i32, i32] + [P] * 10 + [i32, P]
    lib.hs_resolve_spec_layers.restype = ctypes.c_int
    lib.hs_gather_spec.argtypes = [P, i32, P, i32, i32, i32, P]
    lib.hs_gather_spec.restype = ctypes.c_int
    lib.hs_backup_spec.argtypes = [P, i32, i32] + [P] * 5 + [P]
    lib.hs_backup_spec.restype = ctypes.c_int
    lib.hs_gather.restype = ctypes.c_int
    lib.hs_invalidate_tokens.argtypes = [P, i32] + [P] * 5 + [P]
    lib.hs_invalidate_tokens.restype = ctypes.c_int
    lib.hs_invalidate_host_rows.argtypes = [P, i32, P, P, P, i32, P, P, P]
    lib.hs_invalidate_host_rows.restype = ctypes.c_int
    lib.hs_get_error.argtypes = [P, ctypes.POINTER(ctypes.c_uint32), ctypes.c_int]
    lib.hs_get_error.restype = ctypes.c_int
    lib.hs_destroy.argtypes = [P]
    lib.hs_destroy.restype = ctypes.c_int
    lib.hs_status_str.argtypes = [ctypes.c_int]
    lib.hs_status_str.restype = ctypes.c_char_p
    lib.hs_host_register.argtypes = [P, sz, ctypes.POINTER(P)]
    lib.hs_host_register.restype = ctypes.c_int
    lib.hs_host_unregister.argtypes = [P]
    lib.hs_host_unregister.restype = ctypes.c_int
    lib.hs_host_numa_node.argtypes = [i32, ctypes.POINTER(i32)]
    lib.hs_host_numa_node.restype = ctypes.c_int
    lib.hs_host_bind_node.argtypes = [P, sz, i32]
    lib.hs_host_bind_node.restype = ctypes.c_int
    lib.hs_resolve_noalloc.argtypes = [cfgp, P, P, i64, i64, i32] + [P] * 11 + [P]
    lib.hs_resolve_noalloc.restype = ctypes.c_int
    f32, poolp = ctypes.c_float, ctypes.POINTER(hs_page_pool)
    lib.hs_fp4_pack_rows.argtypes = [i32, P, i64, P, f32, P, i64, P, P]
    lib.hs_fp4_unpack_rows.argtypes = [i32, P, i64, P, f32, P, i64, P, P]
    lib.hs_fp4_mla_splits.argtypes = [i32, i32, i32, i64]
    lib.hs_fp4_mla_splits.restype = i32
    lib.hs_fp4_mla_workspace_bytes.argtypes = [i32, i32, i32, i32]
    lib.hs_fp4_mla_workspace_bytes.restype = sz
    lib.hs_fp4_sparse_mla_decode.argtypes = [i32] * 4 + [P, P, i64, P, f32, f32, P, P, P, sz, P, P]
    lib.hs_fp4_window_mla_decode.argtypes = ([i32] * 6 + [P, P, i64, i32, i32, P, P, f32, f32, P, P, P, sz, P, P])
    lib.hs_pages_workspace_bytes.argtypes = [i32, i32]
    lib.hs_pages_workspace_bytes.restype = sz
    lib.hs_pages_init.argtypes = [poolp, P]
    lib.hs_pages_extend.argtypes = [poolp, i32, P, P, P, P, P]
    lib.hs_pages_fork.argtypes = [poolp, i32, P, P, P, P, P]
    lib.hs_pages_free.argtypes = [poolp, i32, P, P, P, P]
    lib.hs_pages_compact.argtypes = [poolp, P]
    lib.hs_batch_plan.argtypes = [i32, P, P, P, i32, P, i32, i32, i64, i32] + [P] * 5 + [i32, P, P, P]
    lib.hs_fp8_pack_rows.argtypes = [i32, P, i64, P, P, f32, P, P, i32, P, i64, P, P]
    lib.hs_fp8_unpack_rows.argtypes = [i32, P, i64, P, P, i64, P, P]
    lib.hs_chunk_mla_workspace_bytes.argtypes = [i32, i32, i32, i64]
    lib.hs_chunk_mla_workspace_bytes.restype = sz
    lib.hs_chunk_mla.argtypes = [i32, i32, i32, P, P, P, P, i64, i32, i32, P, f32, P, P, i64, P, sz, P, P]
    for name in ("hs_batch_plan", "hs_fp8_pack_rows", "hs_fp8_unpack_rows", "hs_chunk_mla",
                 "hs_fp4_pack_rows", "hs_fp4_unpack_rows", "hs_fp4_sparse_mla_decode", "hs_fp4_window_mla_decode",
                 "hs_pages_init", "hs_pages_extend", "hs_pages_fork", "hs_pages_free", "hs_pages_compact"):
        getattr(lib, name).restype = ctypes.c_int
    return lib


class _Lazy:
    """Loads libhs.so on first attribute access (so the build module imports without it)."""

    _cdll = None

    def __getattr__(self, name):
        if _Lazy._cdll is None:
            _Lazy._cdll = _load()
        return getattr(_Lazy._cdll, name)


_lib = _Lazy()


def _addr(x) -> Optional[int]:
    """Raw address of a torch tensor, numpy array or int; None stays None (NULL)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        if not x.is_contiguous():
            raise ValueError("arrays passed to libhs must be contiguous")
        return x.data_ptr()
    if hasattr(x, "ctypes"):
        if not x.flags.c_contiguous:
            raise ValueError("arrays passed to libhs must be contiguous")
        return x.ctypes.data
    raise TypeError(f"cannot take the address of {type(x).__name__}")


_torch = None  # imported with the first tensor
_types = {}  # of a letter: the dtypes that the library can read as it (the first is the one that it is mostly given)
_wants = {}  # of a call's letters: the first dtype of each, None for any


def _import_torch():
    global _torch
    import torch
    _types.update({"i": (torch.int32, torch.uint32), "h": (torch.bfloat16, torch.int16, torch.uint16),
                   "f": (torch.float32,)})
    _torch = torch
    return torch


def _device_check(on: int) -> int:
    """`on`, the device of an array (-1: none), where it is the current device."""
    if on < 0:
        raise ValueError("this argument is read or written on the GPU: pass a CUDA tensor or a device address")
    here = (_torch or _import_torch()).cuda.current_device()
    if on != here:
        raise ValueError(f"the tensor is on cuda:{on}, the current device is cuda:{here}")
    return on


def _type_check(kind: str, dtype) -> None:
    """Elements of the type that the library reads: i 32-bit integers, h bf16 values or their bits, f fp32."""
    if dtype not in _types[kind]:
        wanted = {"i": "32-bit integers", "h": "bf16 values or their 16-bit patterns", "f": "32-bit floats"}[kind]
        raise ValueError(f"{wanted} are needed here, not {dtype}")


def _rows_on_gpu(x, stride: int) -> Optional[int]:
    """_on_gpu of a 2-D array with rows of consecutive bf16 values, `stride` values apart."""
    if x is None or isinstance(x, int):
        return x
    _device_check(x.get_device() if hasattr(x, "get_device") else -1)
    _type_check("h", x.dtype)
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("rows of consecutive values are needed")
    if x.size(0) > 1 and x.stride(0) != stride:
        raise ValueError(f"the rows are {x.stride(0)} values apart, not {stride}")
    return x.data_ptr()


def _on_gpu(kinds: str, *xs, here: int = -1):
    """Addresses of contiguous arrays, which have to be on the current device (`here`, where that is known) and of the
    types in `kinds` (a letter an array, "." any; None and raw addresses are taken as they are). Short, as a call's
    host time is mostly this: 0.4 us an array."""
    wants = _wants.get(kinds)
    if wants is None:
        if all(x is None or isinstance(x, int) for x in xs):
            return xs  # addresses: torch need not be there
        _torch or _import_torch()
        wants = _wants[kinds] = tuple(None if k == "." else _types[k][0] for k in kinds)
    out = []
    for want, x in zip(wants, xs):
        if x is not None and not isinstance(x, int):
            on = x.get_device() if hasattr(x, "get_device") else -1
            if on != here or on < 0:
                here = _device_check(on)
            if want is not None and x.dtype is not want:
                _type_check(kinds[len(out)], x.dtype)
            if not x.is_contiguous():
                raise ValueError("arrays passed to libhs must be contiguous")
            x = x.data_ptr()
        out.append(x)
    return out


def _stream(s) -> Optional[int]:
    if s is None:
        return None
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(status: int, what: str) -> None:
    if status != HS_OK:
        raise HsError(status, what)


def hs_status_str(status: int) -> str:
    return _lib.hs_status_str(status).decode()


def make_config(max_requests: int, top_k: int, hot_slots: int, row_bytes: int, num_layers: int = 1,
                page_size: int = 0, max_context: int = 0, max_pages: int = 0, host_row_stride: int = 0) -> hs_config:
    """host_row_stride: bytes between host rows of one layer (0: row_bytes, one pool per layer;
    num_layers * row_bytes with pools base + l * row_bytes: every layer of a token in one row)."""
    return hs_config(max_requests, top_k, hot_slots, row_bytes, num_layers, page_size, max_context, max_pages,
                     host_row_stride)


def hs_workspace_bytes(cfg: hs_config) -> int:
    return int(_lib.hs_workspace_bytes(ctypes.byref(cfg)))


class Handle:
    """Owns the C handle; the pools, tables and workspace stay the caller's."""

    def __init__(self, ptr: int, cfg: hs_config):
        self.ptr = ptr
        self.cfg = cfg

    def __del__(self):
        if getattr(self, "ptr", None):
            _lib.hs_destroy(self.ptr)
            self.ptr = None


def hs_create(cfg: hs_config, host_pools: Sequence, device_pools: Sequence, host_rows: int, device_rows: int,
              workspace) -> Handle:
    hp = (ctypes.c_void_p * len(host_pools))(*[_addr(p) for p in host_pools])
    dp = (ctypes.c_void_p * len(device_pools))(*[_addr(p) for p in device_pools])
    out = ctypes.c_void_p()
    _check(_lib.hs_create(ctypes.byref(cfg), hp if len(host_pools) else None, dp if len(device_pools) else None,
                          host_rows, device_rows, _addr(workspace), ctypes.byref(out)), "hs_create")
    return Handle(out.value, cfg)


def hs_resolve(h: Handle, num_requests: int, top_k_tokens, seq_lens, host_cache_locs, device_buffer_locs,
               device_buffer_tokens, lru_slots, lru_clock, resident_pages, out_rows, miss_counts,
               stream=None) -> None:
    _check(_lib.hs_resolve(h.ptr if h else None, num_requests, _addr(top_k_tokens), _addr(seq_lens),
                           _addr(host_cache_locs), _addr(device_buffer_locs), _addr(device_buffer_tokens),
                           _addr(lru_slots), _addr(lru_clock), _addr(resident_pages), _addr(out_rows),
                           _addr(miss_counts), _stream(stream)), "hs_resolve")


def hs_resolve_layers(h: Handle, num_requests: int, top_k_tokens, seq_lens, host_cache_locs, device_buffer_locs,
                      device_buffer_tokens, lru_slots, lru_clock, resident_pages, out_rows, miss_counts,
                      copy_layers: int, stream=None) -> None:
    _check(_lib.hs_resolve_layers(h.ptr if h else None, num_requests, _addr(top_k_tokens), _addr(seq_lens),
                                  _addr(host_cache_locs), _addr(device_buffer_locs), _addr(device_buffer_tokens),
                                  _addr(lru_slots), _addr(lru_clock), _addr(resident_pages), _addr(out_rows),
                                  _addr(miss_counts), copy_layers, _stream(stream)), "hs_resolve_layers")


def hs_resolve_spec(h: Handle, num_requests: int, num_queries: int, top_k_tokens, committed_lens, host_cache_locs,
                    device_buffer_locs, device_buffer_tokens, lru_slots, lru_clock, resident_pages, out_rows,
                    miss_counts, stream=None) -> None:
    _check(_lib.hs_resolve_spec(h.ptr if h else None, num_requests, num_queries, _addr(top_k_tokens),
                                _addr(committed_lens), _addr(host_cache_locs), _addr(device_buffer_locs),
                                _addr(device_buffer_tokens), _addr(lru_slots), _addr(lru_clock),
                                _addr(resident_pages), _addr(out_rows), _addr(miss_counts), _stream(stream)),
           "hs_resolve_spec")


def hs_resolve_spec_layers(h: Handle, num_requests: int, num_queries: int, top_k_tokens, committed_lens,
                           host_cache_locs, device_buffer_locs, device_buffer_tokens, lru_slots, lru_clock,
                           resident_pages, out_rows, miss_counts, copy_layers: int, stream=None) -> None:
    _check(_lib.hs_resolve_spec_layers(h.ptr if h else None, num_requests, num_queries, _addr(top_k_tokens),
                                       _addr(committed_lens), _addr(host_cache_locs), _addr(device_buffer_locs),
                                       _addr(device_buffer_tokens), _addr(lru_slots), _addr(lru_clock),
                                       _addr(resident_pages), _addr(out_rows), _addr(miss_counts), copy_layers,
                                       _stream(stream)), "hs_resolve_spec_layers")


def hs_gather_spec(h: Handle, num_requests: int, host_cache_locs, query: int, first_layer: int, num_layers: int,
                   stream=None) -> None:
    _check(_lib.hs_gather_spec(h.ptr if h else None, num_requests, _addr(host_cache_locs), query, first_layer,
                               num_layers, _stream(stream)), "hs_gather_spec")


def hs_backup_spec(h: Handle, num_requests: int, num_queries: int, committed_lens, accepted, host_cache_locs,
                   device_buffer_locs, resident_pages, stream=None) -> None:
    _check(_lib.hs_backup_spec(h.ptr if h else None, num_requests, num_queries, _addr(committed_lens),
                               _addr(accepted), _addr(host_cache_locs), _addr(device_buffer_locs),
                               _addr(resident_pages), _stream(stream)), "hs_backup_spec")


def hs_gather(h: Handle, num_requests: int, host_cache_locs, first_layer: int, num_layers: int,
              stream=None) -> None:
    _check(_lib.hs_gather(h.ptr if h else None, num_requests, _addr(host_cache_locs), first_layer, num_layers,
                          _stream(stream)), "hs_gather")


def hs_backup(h: Handle, num_requests: int, seq_lens, host_cache_locs, device_buffer_locs, resident_pages,
              stream=None) -> None:
    _check(_lib.hs_backup(h.ptr if h else None, num_requests, _addr(seq_lens), _addr(host_cache_locs),
                          _addr(device_buffer_locs), _addr(resident_pages), _stream(stream)), "hs_backup")


def hs_invalidate_tokens(h: Handle, num_requests: int, seq_lens, token_offsets, tokens, device_buffer_tokens,
                         lru_slots, stream=None) -> None:
    _check(_lib.hs_invalidate_tokens(h.ptr if h else None, num_requests, _addr(seq_lens), _addr(token_offsets),
                                     _addr(tokens), _addr(device_buffer_tokens), _addr(lru_slots),
                                     _stream(stream)), "hs_invalidate_tokens")


def hs_invalidate_host_rows(h: Handle, num_requests: int, seq_lens, host_cache_locs, rows, n: int,
                            device_buffer_tokens, lru_slots, stream=None) -> None:
    _check(_lib.hs_invalidate_host_rows(h.ptr if h else None, num_requests, _addr(seq_lens), _addr(host_cache_locs),
                                        _addr(rows), n, _addr(device_buffer_tokens), _addr(lru_slots),
                                        _stream(stream)), "hs_invalidate_host_rows")


def hs_sparse_mla_workspace_bytes(num_requests: int, num_heads: int, splits: int) -> int:
    return int(_lib.hs_sparse_mla_workspace_bytes(num_requests, num_heads, splits))


def hs_sparse_mla_launches(num_requests: int, num_heads: int, splits: int) -> int:
    """Kernel launches of one hs_sparse_mla_decode call of this shape on the current device."""
    return int(_lib.hs_sparse_mla_launches(num_requests, num_heads, splits))


def hs_sparse_mla_decode(num_requests: int, num_heads: int, top_k: int, splits: int, q, kv_pool, pool_rows: int,
                         out_rows, sm_scale: float, o, lse, workspace, workspace_bytes: int, error_flags,
                         stream=None) -> None:
    _check(_lib.hs_sparse_mla_decode(num_requests, num_heads, top_k, splits, _addr(q), _addr(kv_pool), pool_rows,
                                     _addr(out_rows), float(sm_scale), _addr(o), _addr(lse), _addr(workspace),
                                     workspace_bytes, _addr(error_flags), _stream(stream)), "hs_sparse_mla_decode")


def hs_fp4_pack_rows(n: int, kv, kv_stride: int, rows, latent_scale: float, pool, pool_rows: int, error_flags,
                     stream=None) -> None:
    """Quantise n tokens (bf16 [n, kv_stride], 576 used) into the 4-bit rows `rows` of the pool."""
    kv = _rows_on_gpu(kv, kv_stride)
    rows, pool, error_flags = _on_gpu("i.i", rows, pool, error_flags)
    _check(_lib.hs_fp4_pack_rows(n, kv, kv_stride, rows, latent_scale, pool, pool_rows, error_flags, _stream(stream)),
           "hs_fp4_pack_rows")


def hs_fp4_unpack_rows(n: int, pool, pool_rows: int, rows, latent_scale: float, kv, kv_stride: int, error_flags,
                       stream=None) -> None:
    """Read the 4-bit rows `rows` back as bf16 into kv ([n, kv_stride], 576 written)."""
    kv = _rows_on_gpu(kv, kv_stride)
    pool, rows, error_flags = _on_gpu(".ii", pool, rows, error_flags)
    _check(_lib.hs_fp4_unpack_rows(n, pool, pool_rows, rows, latent_scale, kv, kv_stride, error_flags,
                                   _stream(stream)), "hs_fp4_unpack_rows")


def hs_fp4_mla_splits(num_requests: int, num_heads: int, num_queries: int, rows: int) -> int:
    """Splits that suit a call over up to `rows` rows per request on the current device."""
    return int(_lib.hs_fp4_mla_splits(num_requests, num_heads, num_queries, rows))


def hs_fp4_mla_workspace_bytes(num_requests: int, num_heads: int, num_queries: int, splits: int) -> int:
    return int(_lib.hs_fp4_mla_workspace_bytes(num_requests, num_heads, num_queries, splits))


def hs_fp4_sparse_mla_decode(num_requests: int, num_heads: int, top_k: int, splits: int, q, kv_pool, pool_rows: int,
                             out_rows, sm_scale: float, latent_scale: float, o, lse, workspace, workspace_bytes: int,
                             error_flags, stream=None) -> None:
    q, kv_pool, out_rows, o, lse, workspace, error_flags = _on_gpu("h.ihf.i", q, kv_pool, out_rows, o, lse, workspace,
                                                                   error_flags)
    _check(_lib.hs_fp4_sparse_mla_decode(num_requests, num_heads, top_k, splits, q, kv_pool, pool_rows, out_rows,
                                         sm_scale, latent_scale, o, lse, workspace, workspace_bytes, error_flags,
                                         _stream(stream)), "hs_fp4_sparse_mla_decode")


def hs_fp4_window_mla_decode(num_requests: int, num_heads: int, num_queries: int, window: int, sinks: int,
                             splits: int, q, kv_pool, pool_rows: int, page_size: int, max_pages: int, seq_lens,
                             resident_pages, sm_scale: float, latent_scale: float, o, lse, workspace,
                             workspace_bytes: int, error_flags, stream=None) -> None:
    q, kv_pool, seq_lens, resident_pages, o, lse, workspace, error_flags = _on_gpu(
        "h.iihf.i", q, kv_pool, seq_lens, resident_pages, o, lse, workspace, error_flags)
    _check(_lib.hs_fp4_window_mla_decode(num_requests, num_heads, num_queries, window, sinks, splits, q, kv_pool,
                                         pool_rows, page_size, max_pages, seq_lens, resident_pages, sm_scale,
                                         latent_scale, o, lse, workspace, workspace_bytes, error_flags,
                                         _stream(stream)), "hs_fp4_window_mla_decode")


def hs_pages_workspace_bytes(num_requests: int, num_pages: int) -> int:
    return int(_lib.hs_pages_workspace_bytes(num_requests, num_pages))


def make_page_pool(device_pools: Sequence, num_requests: int, max_pages: int, num_pages: int, page_size: int,
                   row_bytes: int, resident_pages, page_refs, free_pages, free_count, workspace, workspace_bytes: int,
                   error_flags) -> hs_page_pool:
    """The descriptor of the hs_pages_* calls. It keeps the tensors that it points to alive."""
    if not 1 <= len(device_pools) <= HS_MAX_LAYERS:
        raise ValueError(f"1 to {HS_MAX_LAYERS} device pools")
    arrays = _on_gpu("iiiii.", resident_pages, page_refs, free_pages, free_count, error_flags, workspace)
    p = hs_page_pool(num_requests, max_pages, num_pages, page_size, row_bytes, len(device_pools),
                     (ctypes.c_void_p * HS_MAX_LAYERS)(*_on_gpu("." * len(device_pools), *device_pools)), *arrays, workspace_bytes)
    p.kept = (list(device_pools), resident_pages, page_refs, free_pages, free_count, error_flags, workspace)
    p.device = next((x.get_device() for x in (*device_pools, *p.kept[1:]) if hasattr(x, "get_device")), None)
    return p


def _pool_here(pool: Optional[hs_page_pool]) -> int:
    """The pool's device, which has to be the current one; -1 if it has none."""
    return -1 if pool is None or pool.device is None else _device_check(pool.device)


def hs_pages_init(pool: hs_page_pool, stream=None) -> None:
    _pool_here(pool)
    _check(_lib.hs_pages_init(pool, _stream(stream)), "hs_pages_init")


def hs_pages_extend(pool: hs_page_pool, n: int, requests, old_lens, new_lens, granted=None, stream=None) -> None:
    arrays = _on_gpu("iiii", requests, old_lens, new_lens, granted, here=_pool_here(pool))
    _check(_lib.hs_pages_extend(pool, n, *arrays, _stream(stream)), "hs_pages_extend")


def hs_pages_fork(pool: hs_page_pool, n: int, parents, children, lens, granted=None, stream=None) -> None:
    arrays = _on_gpu("iiii", parents, children, lens, granted, here=_pool_here(pool))
    _check(_lib.hs_pages_fork(pool, n, *arrays, _stream(stream)), "hs_pages_fork")


def hs_pages_free(pool: hs_page_pool, n: int, requests, first_pages=None, end_pages=None, stream=None) -> None:
    arrays = _on_gpu("iii", requests, first_pages, end_pages, here=_pool_here(pool))
    _check(_lib.hs_pages_free(pool, n, *arrays, _stream(stream)), "hs_pages_free")


def hs_pages_compact(pool: hs_page_pool, stream=None) -> None:
    _pool_here(pool)
    _check(_lib.hs_pages_compact(pool, _stream(stream)), "hs_pages_compact")


def hs_batch_plan(n: int, requests, old_lens, new_lens, num_requests: int, resident_pages, max_pages: int,
                  page_size: int, pool_rows: int, max_tokens: int, token_offsets, seq_lens, entries, positions, rows,
                  max_blocks: int, block_tables, error_flags, stream=None) -> None:
    """A step's flat tokens, their positions and pool rows, and the entries' block tables."""
    (requests, old_lens, new_lens, resident_pages, token_offsets, seq_lens, entries, positions, rows, block_tables,
     error_flags) = _on_gpu("iiiiiiiiiii", requests, old_lens, new_lens, resident_pages, token_offsets, seq_lens, entries,
                            positions, rows, block_tables, error_flags)
    _check(_lib.hs_batch_plan(n, requests, old_lens, new_lens, num_requests, resident_pages, max_pages, page_size,
                              pool_rows, max_tokens, token_offsets, seq_lens, entries, positions, rows, max_blocks,
                              block_tables, error_flags, _stream(stream)), "hs_batch_plan")


def hs_fp8_pack_rows(n: int, kv, kv_stride: int, rows, norm_weight, norm_eps: float, positions, rope_table,
                     rope_positions: int, pool, pool_rows: int, error_flags, stream=None) -> None:
    """Normalise, rotate and quantise n tokens (bf16 [n, kv_stride], 576 used) into the fp8 rows `rows` of the pool."""
    kv = _rows_on_gpu(kv, kv_stride)
    rows, norm_weight, positions, rope_table, pool, error_flags = _on_gpu("ihif.i", rows, norm_weight, positions,
                                                                          rope_table, pool, error_flags)
    _check(_lib.hs_fp8_pack_rows(n, kv, kv_stride, rows, norm_weight, norm_eps, positions, rope_table, rope_positions,
                                 pool, pool_rows, error_flags, _stream(stream)), "hs_fp8_pack_rows")


def hs_fp8_unpack_rows(n: int, pool, pool_rows: int, rows, kv, kv_stride: int, error_flags, stream=None) -> None:
    """Read the fp8 rows `rows` back as bf16 into kv ([n, kv_stride], 576 written)."""
    kv = _rows_on_gpu(kv, kv_stride)
    pool, rows, error_flags = _on_gpu(".ii", pool, rows, error_flags)
    _check(_lib.hs_fp8_unpack_rows(n, pool, pool_rows, rows, kv, kv_stride, error_flags, _stream(stream)),
           "hs_fp8_unpack_rows")


def hs_chunk_mla_workspace_bytes(n: int, num_heads: int, max_tokens: int, max_kv_tokens: int) -> int:
    return int(_lib.hs_chunk_mla_workspace_bytes(n, num_heads, max_tokens, max_kv_tokens))


def hs_chunk_mla(n: int, num_heads: int, max_tokens: int, token_offsets, seq_lens, q, kv_pool, pool_rows: int,
                 page_size: int, max_blocks: int, block_tables, sm_scale: float, o, lse, max_kv_tokens: int, workspace,
                 workspace_bytes: int, error_flags, stream=None) -> None:
    """Causal attention of the batch's new tokens over the pages of their sequences."""
    token_offsets, seq_lens, q, kv_pool, block_tables, o, lse, workspace, error_flags = _on_gpu(
        "iih.ihf.i", token_offsets, seq_lens, q, kv_pool, block_tables, o, lse, workspace, error_flags)
    _check(_lib.hs_chunk_mla(n, num_heads, max_tokens, token_offsets, seq_lens, q, kv_pool, pool_rows, page_size,
                             max_blocks, block_tables, sm_scale, o, lse, max_kv_tokens, workspace, workspace_bytes,
                             error_flags, _stream(stream)), "hs_chunk_mla")


def hs_reset_hints(h: Handle, stream=None) -> None:
    _check(_lib.hs_reset_hints(h.ptr if h else None, _stream(stream)), "hs_reset_hints")


def hs_launch_shape(h: Handle):
    """(copy CTAs per request, kernel launches per hs_resolve) chosen by hs_create."""
    c, n = ctypes.c_int32(0), ctypes.c_int32(0)
    _check(_lib.hs_launch_shape(h.ptr if h else None, ctypes.byref(c), ctypes.byref(n)), "hs_launch_shape")
    return int(c.value), int(n.value)


def hs_get_error(h: Handle, clear: bool = False) -> int:
    """The sticky HS_FLAG_* word (synchronises the device)."""
    flags = ctypes.c_uint32(0)
    st = _lib.hs_get_error(h.ptr, ctypes.byref(flags), 1 if clear else 0)
    if st not in (HS_OK, HS_ERR_DEVICE_FLAGGED):
        raise HsError(st, "hs_get_error")
    return int(flags.value)


def hs_destroy(h: Handle) -> None:
    if h and h.ptr:
        _check(_lib.hs_destroy(h.ptr), "hs_destroy")
        h.ptr = None


def hs_host_register(host_array, nbytes: Optional[int] = None) -> int:
    """Pin and map a host range for the kernels; returns its device-side address."""
    ptr = _addr(host_array)
    if nbytes is None:
        nbytes = host_array.nbytes
    dev = ctypes.c_void_p()
    _check(_lib.hs_host_register(ptr, nbytes, ctypes.byref(dev)), "hs_host_register")
    return int(dev.value)


def hs_host_unregister(host_array) -> None:
    _check(_lib.hs_host_unregister(_addr(host_array)), "hs_host_unregister")


def hs_host_numa_node(device: int) -> int:
    """The host memory node nearest `device`, or -1 when the platform does not say."""
    n = ctypes.c_int32(-1)
    _check(_lib.hs_host_numa_node(device, ctypes.byref(n)), "hs_host_numa_node")
    return int(n.value)


def hs_host_bind_node(addr, nbytes: int, node: int) -> None:
    """Prefer memory node `node` for the untouched pages of [addr, addr + nbytes)."""
    _check(_lib.hs_host_bind_node(_addr(addr), nbytes, node), "hs_host_bind_node")


def hs_resolve_noalloc(cfg: hs_config, host_pools: Sequence, device_pools: Sequence, host_rows: int,
                       device_rows: int, num_requests: int, top_k_tokens, seq_lens, host_cache_locs,
                       device_buffer_locs, device_buffer_tokens, lru_slots, lru_clock, resident_pages, out_rows,
                       miss_counts, error_flags=None, stream=None) -> None:
    """hs_resolve without a handle or workspace, for callers that cannot allocate device
    memory: the library keeps the scratch in its own device array (see include/hs.h)."""
    hp = (ctypes.c_void_p * len(host_pools))(*[_addr(p) for p in host_pools])
    dp = (ctypes.c_void_p * len(device_pools))(*[_addr(p) for p in device_pools])
    _check(_lib.hs_resolve_noalloc(ctypes.byref(cfg), hp if len(host_pools) else None,
                                   dp if len(device_pools) else None, host_rows, device_rows, num_requests,
                                   _addr(top_k_tokens), _addr(seq_lens), _addr(host_cache_locs),
                                   _addr(device_buffer_locs), _addr(device_buffer_tokens), _addr(lru_slots),
                                   _addr(lru_clock), _addr(resident_pages), _addr(out_rows), _addr(miss_counts),
                                   _addr(error_flags), _stream(stream)), "hs_resolve_noalloc")
