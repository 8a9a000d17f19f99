"""Paged KV-cache attention for GB300 (sm_103a): Python binding of ``libkvc.so``.

Every function here marshals arguments (tensor pointers, sizes, the current
CUDA stream) and calls the C ABI of the same name declared in
``include/kvc.h``; all arithmetic runs in the library's CUDA kernels or its
native host code.  There is no fallback: if the library has not been built
(``paged_kv_cache_27_gb300.build()``), importing this package raises.

PyTorch provides device memory and streams only.
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass
from typing import Optional, Sequence

import numpy as np
import torch  # loads the CUDA runtime that libkvc.so links against
from torch.multiprocessing.reductions import StorageWeakRef

from ._build import LIB as _LIB_PATH
from ._build import build

__all__ = [
    "KvcError", "KvcConfig", "KVC_F16", "KVC_F32", "build", "lib_path",
    "kvc_version", "kvc_set_checked_mode", "kvc_device_error_flags", "kv_cache_pool_bytes",
    "kv_cache_create", "kv_cache_destroy", "kv_cache_layer", "kv_block_alloc", "kv_block_share",
    "kv_block_release", "kv_block_refcount", "kv_block_num_free", "kv_cache_utilisation",
    "kv_block_cow", "kv_copy_blocks", "kv_slot_mapping", "kv_step_prepare", "kv_append",
    "paged_decode_plan", "paged_decode_workspace_init", "paged_decode_attention",
    "paged_decode_append_attention", "kvc_set_launch_overlap", "kvc_set_cascade_min_saved_blocks", "kvc_set_multi_tc", "kvc_copy_async", "KVC_COPY_AHEAD", "PreparedCall",
    "kvc_trace_read",
    "paged_decode_attention_static_workspace", "paged_decode_cascade_plan", "paged_decode_cascade_attention", "kv_cascade_groups",
    "paged_decode_multi_plan", "paged_decode_multi_attention", "kv_append_fp8", "paged_decode_attention_fp8",
    "kv_fp8_record_bytes",
    "prefill_attention", "prefill_attention_ex", "fp8_v_position", "DEVERR",
    "kv_tree_masks", "kv_rope_turns", "kv_append_rope", "paged_decode_tree_plan", "paged_decode_tree_attention",
    "draft_tree_verify", "kv_tree_commit",
    "kv_block_tables", "kv_append_fp8_block", "paged_decode_fp8_block_plan", "paged_decode_attention_fp8_block",
    "paged_decode_window_plan", "paged_decode_window_attention", "prefill_window_attention",
]

KVC_F16, KVC_F32 = 0, 1
KVC_PREFILL_P_F16, KVC_PREFILL_P_SPLIT = 0, 1
STATUS = {0: "KVC_OK", 1: "KVC_ERR_INVALID", 2: "KVC_ERR_OOM", 3: "KVC_ERR_CAPACITY", 4: "KVC_ERR_CUDA",
          5: "KVC_ERR_UNSUPPORTED"}
DEVERR = {"BLOCK_ID": 0x1, "CONTEXT": 0x2, "SLOT": 0x4, "TIMEOUT": 0x8, "SEQLENS": 0x10, "TREE": 0x20,
          "BLOCKS": 0x40}


class KvcError(RuntimeError):
    def __init__(self, status: int, func: str, msg: str):
        self.status = status
        self.name = STATUS.get(status, str(status))
        super().__init__(f"{func}: {self.name}: {msg}")


class _Config(ctypes.Structure):
    _fields_ = [("num_layers", ctypes.c_int), ("num_blocks", ctypes.c_int), ("block_size", ctypes.c_int),
                ("num_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("dtype", ctypes.c_int)]


@dataclass
class KvcConfig:
    num_layers: int
    num_blocks: int
    num_kv_heads: int
    head_dim: int
    block_size: int = 16
    dtype: int = KVC_F16

    def _c(self) -> _Config:
        return _Config(self.num_layers, self.num_blocks, self.block_size, self.num_kv_heads, self.head_dim,
                       self.dtype)

    @property
    def pool_shape(self):
        return (self.num_layers, self.num_blocks, self.num_kv_heads, self.block_size, self.head_dim)


def lib_path() -> str:
    return _LIB_PATH


def _load():
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"libkvc.so is not built ({_LIB_PATH}); run paged_kv_cache_27_gb300.build()")
    lib = ctypes.CDLL(_LIB_PATH)
    P, I, I32, I64, SZ, D = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t,
                             ctypes.c_double)
    PI32, PI64, PSZ, PI = (ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int64),
                           ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_int))
    sig = {
        "kvc_last_error_string": (ctypes.c_char_p, []),
        "kvc_version": (I, []),
        "kvc_set_checked_mode": (I, [I]),
        "kvc_device_error_flags": (I, [ctypes.POINTER(ctypes.c_uint32), I]),
        "kv_cache_pool_bytes": (I, [ctypes.POINTER(_Config), PSZ]),
        "kv_cache_create": (I, [ctypes.POINTER(_Config), P, P, ctypes.POINTER(P)]),
        "kv_cache_destroy": (I, [P]),
        "kv_cache_layer": (I, [P, I, ctypes.POINTER(P), ctypes.POINTER(P)]),
        "kv_block_alloc": (I, [P, PI32]),
        "kv_block_share": (I, [P, I32]),
        "kv_block_release": (I, [P, I32]),
        "kv_block_refcount": (I, [P, I32, PI32]),
        "kv_block_num_free": (I, [P, PI32]),
        "kv_cache_utilisation": (I, [P, ctypes.POINTER(D)]),
        "kv_block_cow": (I, [P, I32, PI32, P]),
        "kv_copy_blocks": (I, [P, P, P, I, P]),
        "kv_slot_mapping": (I, [P, I, I, P, P, I, P]),
        "kv_step_prepare": (I, [P, P, I, P, P, I, P, P, P, PI]),
        "kv_append": (I, [P, I, P, P, P, I, P]),
        "paged_decode_plan": (I, [I, I, I, I, I, I, I, PI, PI, PSZ]),
        "paged_decode_workspace_init": (I, [P, SZ, P]),
        "paged_decode_attention": (I, [P, P, P, I, P, I, P, I, I, I, I, I, I, ctypes.c_float, P, I, P, SZ, I, P]),
        "paged_decode_append_attention": (I, [P, P, P, P, P, I, P, I, P, I, I, I, I, I, I, ctypes.c_float, P,
                                              I, P, SZ, I, P]),
        "kvc_set_launch_overlap": (I, [I]),
        "kvc_set_cascade_min_saved_blocks": (I, [I]),
        "kvc_set_multi_tc": (I, [I]),
        "kvc_copy_async": (I, [P, P, SZ, ctypes.c_uint, P]),
        "paged_decode_attention_static_workspace": (I, [P, P, P, I, P, I, P, I, I, I, I, I, I, ctypes.c_float, P, I,
                                                        I, P]),
        "kvc_trace_read": (I, [P, I, PI, I]),
        "paged_decode_cascade_plan": (I, [I, I, I, I, I, I, I, I, PSZ]),
        "kv_cascade_groups": (I, [P, I, I, P, I, I, P, PI, P, PI]),
        "paged_decode_multi_plan": (I, [I, I, I, I, I, I, I, PSZ]),
        "kv_fp8_record_bytes": (I, [I, PSZ]),
        "kv_append_fp8": (I, [P, P, P, I, P, I, I, I, I, P]),
        "paged_decode_attention_fp8": (I, [P, P, I, P, I, P, I, I, I, I, I, I, ctypes.c_float, P, I, P, SZ, I, P]),
        "paged_decode_multi_attention": (I, [P, P, P, I, P, I, P, I, I, I, I, I, I, I, ctypes.c_float, P, I, P, SZ,
                                             P]),
        "paged_decode_cascade_attention": (I, [P, P, P, I, P, I, P, P, P, I, I, I, I, I, I, I, I, ctypes.c_float, P,
                                               I, P, SZ, P]),
        "kv_tree_masks": (I, [P, P, I, I, P, P]),
        "kv_rope_turns": (I, [P, I, P]),
        "kv_append_rope": (I, [P, I64, P, I64, P, I64, I, I, I, I, P, P, ctypes.c_float, P, I, I, P, P, P, P, P, P, I,
                               I, P, P]),
        "paged_decode_tree_plan": (I, [I, I, I, I, I, I, I, PSZ]),
        "paged_decode_tree_attention": (I, [P, P, P, I, P, I, P, P, P, I, I, I, I, I, I, I, ctypes.c_float, P, I, P,
                                            SZ, P]),
        "draft_tree_verify": (I, [P, I64, P, I64, I, P, P, P, P, I, I, I, I, P, P, P, P]),
        "kv_tree_commit": (I, [P, P, I, P, P, P, P, I, I, P, P]),
        "kv_block_tables": (I, [P, P, I, P, I, P, I, I, P, I, I, P, P, P, P, I, P]),
        "kv_append_fp8_block": (I, [P, I64, P, I64, I, P, P, P, I, I, I, I, P]),
        "paged_decode_fp8_block_plan": (I, [I, I, I, I, I, I, I, I, PSZ]),
        "paged_decode_attention_fp8_block": (I, [P, P, P, I, P, I, P, I, I, I, I, I, I, I, I, ctypes.c_float, P, I, P,
                                                 SZ, P]),
        "paged_decode_window_plan": (I, [I, I, I, I, I, I, I, I, PSZ]),
        "paged_decode_window_attention": (I, [P, P, P, P, P, I, P, I, P, I, I, I, I, I, I, I, I, ctypes.c_float, P, I,
                                              P, SZ, P]),
        "prefill_window_attention": (I, [P, P, P, P, I, I, I, I, I, I, ctypes.c_float, I, I, I, P, I, P]),
        "kvc_call": (I, [I, ctypes.c_char_p, I, P]),
        "prefill_attention": (I, [P, P, P, P, I, I, I, I, I, I, ctypes.c_float, I, P, I, P]),
        "prefill_attention_ex": (I, [P, P, P, P, I, I, I, I, I, I, ctypes.c_float, I, I, P, I, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()


def _check(status: int, func: str):
    if status != 0:
        raise KvcError(status, func, _lib.kvc_last_error_string().decode(errors="replace"))


# the current stream of a device as a raw handle, without building a torch.cuda.Stream object (a few µs per call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, *tensors) -> Optional[int]:
    if stream is not None:
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    for t in tensors:
        if isinstance(t, torch.Tensor) and t.is_cuda:
            if _raw_stream is not None:
                return _raw_stream(t.get_device())
            return torch.cuda.current_stream(t.device).cuda_stream
    return None


def _dptr(t: Optional[torch.Tensor], dtype=None, name="tensor") -> Optional[int]:
    if t is None:
        return None
    # the common case in one expression (dtypes are singletons); the checks below only name the failure
    if isinstance(t, torch.Tensor) and t.is_cuda and (dtype is None or t.dtype is dtype) and t.is_contiguous():
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be contiguous")


class PreparedCall:
    """One library call whose arguments were checked and converted once (the `prepare=True` form of a launching
    call): calling it launches that call again, on `stream` or else the current stream of the call's device.  It
    keeps its tensors alive; their contents may change between launches, their storage must stay where it is.
    Saves the per-call checks and conversions (~5 µs of host time per decode call)."""
    __slots__ = ("_fn", "_args", "_name", "_device", "_keep")

    def __init__(self, fn, args, name, device, keep):
        self._fn, self._name, self._device, self._keep = fn, name, device, keep
        self._args = tuple(a if a is None else at(a) for a, at in zip(args, fn.argtypes))

    def __call__(self, stream=None) -> None:
        if stream is not None:
            st = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        elif _raw_stream is not None:
            st = _raw_stream(self._device)
        else:
            st = torch.cuda.current_stream(self._device).cuda_stream
        _check(self._fn(*self._args, st), self._name)


class _PreparedCacheCall(PreparedCall):
    """A PreparedCall that holds a cache's handle: it keeps the pools alive too, and refuses after kv_cache_destroy."""
    __slots__ = ("_cache",)

    def __init__(self, fn, args, name, device, keep, cache):
        super().__init__(fn, args, name, device, keep + tuple(cache.pools()))
        self._cache = cache

    def __call__(self, stream=None) -> None:
        if not self._cache.open:
            raise ValueError(f"{self._name}: the cache of this call was destroyed")
        super().__call__(stream)


def _launch(fn, args, name, stream, prepare, keep):
    """Launch fn(*args, stream), or return it as a PreparedCall; keep[0] is a CUDA tensor of the call."""
    if prepare:
        return PreparedCall(fn, args, name, keep[0].get_device(), keep)
    _check(fn(*args, _stream(stream, keep[0])), name)
    return None


def _host(a, dtype) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(a), dtype=dtype)


def _np_ptr(a: np.ndarray) -> int:
    return a.ctypes.data


# ---------------------------------------------------------------- diagnostics
def kvc_version() -> int:
    return _lib.kvc_version()


def kvc_set_checked_mode(on: bool) -> None:
    _check(_lib.kvc_set_checked_mode(int(bool(on))), "kvc_set_checked_mode")


def kvc_set_cascade_min_saved_blocks(blocks: int) -> None:
    """Cascade calls saving fewer than `blocks` block reads per KV head ((B - n_groups) * max_shared_blocks) run the
    plain decode (0: always the cascade kernels)."""
    _check(_lib.kvc_set_cascade_min_saved_blocks(int(blocks)), "kvc_set_cascade_min_saved_blocks")


def kvc_set_multi_tc(on: bool) -> None:
    """Multi-token calls at head dim 64 with up to 64 query rows on the tensor-core kernel (off: the mma.sync kernel)."""
    _check(_lib.kvc_set_multi_tc(int(bool(on))), "kvc_set_multi_tc")


def kvc_set_launch_overlap(on: bool) -> None:
    """Launch decode kernels as programmatic dependents of the previous kernel (see include/kvc.h).  While it is on,
    something (a kernel, a copy, an event) goes between a call that writes a decode call's cache rows, block table or
    lengths, kv_append_rope and kv_tree_commit among them, and that decode call."""
    _check(_lib.kvc_set_launch_overlap(int(bool(on))), "kvc_set_launch_overlap")


KVC_COPY_AHEAD = 1


def _stage_ptr(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not (t.is_cuda or t.device.type == "cpu"):
        raise ValueError(f"{name} must be a CUDA tensor or a pinned CPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def kvc_copy_async(dst: torch.Tensor, src: torch.Tensor, ahead: bool = False, stream=None, prepare: bool = False):
    """Copy src's bytes into dst with the library's staging kernel (see include/kvc.h for the two orderings).

    Each of dst and src is a CUDA tensor or a pinned CPU tensor; both hold the same number of bytes, a multiple
    of 16, at 16-byte aligned addresses.  prepare=True returns a PreparedCall instead of launching."""
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != nbytes:
        raise ValueError("dst and src must hold the same number of bytes")
    args = (_stage_ptr(dst, "dst"), _stage_ptr(src, "src"), nbytes, KVC_COPY_AHEAD if ahead else 0)
    if prepare:
        cuda = dst if dst.is_cuda else src
        return PreparedCall(_lib.kvc_copy_async, args, "kvc_copy_async",
                            cuda.get_device() if cuda.is_cuda else torch.cuda.current_device(), (dst, src))
    _check(_lib.kvc_copy_async(*args, _stream(stream, dst, src)), "kvc_copy_async")


TRACE_DTYPE = np.dtype([("t", "<u8", (8,)), ("seq", "<u4"), ("smid", "<u4"), ("x", "<u4"), ("yz", "<u4")])


def kvc_trace_read(capacity: int = 1 << 16, clear: bool = True) -> np.ndarray:
    """Decode-kernel timeline records (library built with -DKVC_TRACE=1)."""
    buf = np.zeros(capacity, dtype=TRACE_DTYPE)
    n = ctypes.c_int(0)
    _check(_lib.kvc_trace_read(_np_ptr(buf), capacity, ctypes.byref(n), int(bool(clear))), "kvc_trace_read")
    return buf[:n.value]


def kvc_device_error_flags(clear: bool = False) -> int:
    v = ctypes.c_uint32(0)
    _check(_lib.kvc_device_error_flags(ctypes.byref(v), int(bool(clear))), "kvc_device_error_flags")
    return v.value


# ------------------------------------------------------------ cache / pool
def kv_cache_pool_bytes(cfg: KvcConfig) -> int:
    n = ctypes.c_size_t(0)
    c = cfg._c()
    _check(_lib.kv_cache_pool_bytes(ctypes.byref(c), ctypes.byref(n)), "kv_cache_pool_bytes")
    return n.value


class _Cache:
    """What stands behind a handle of kv_cache_create: whether it is open, its pools' device, and their storages, which it
    does not keep alive (they are the caller's)."""
    __slots__ = ("open", "device", "_pools")

    def __init__(self, pools):
        self.open, self._pools = True, [StorageWeakRef(t.untyped_storage()) for t in pools]
        self.device = pools[0].get_device() if pools else None

    def pools(self):
        """The pools' storages, to be kept alive."""
        return [torch.UntypedStorage._new_with_weak_ptr(p.cdata) for p in self._pools]


_caches: dict = {}  # by handle, until kv_cache_destroy


def _open_cache(h: int) -> _Cache:
    cache = _caches.get(h)
    if cache is None:
        raise ValueError("h is not an open cache of kv_cache_create")
    for p in cache._pools:
        if p.expired():
            raise ValueError("the cache's pools are freed")
    return cache


def kv_cache_create(cfg: KvcConfig, k_pool: Optional[torch.Tensor] = None,
                    v_pool: Optional[torch.Tensor] = None) -> int:
    """Handle over caller-owned pools (fp16 [L][NB][Hkv][bs][D]); None, None = host-only pool."""
    if (k_pool is None) != (v_pool is None):
        raise ValueError("k_pool and v_pool: both or neither")
    if k_pool is not None:
        if k_pool.device != v_pool.device:
            raise ValueError("k_pool and v_pool are on several devices")
        need = kv_cache_pool_bytes(cfg)
        for t, nm in ((k_pool, "k_pool"), (v_pool, "v_pool")):
            if t.numel() * t.element_size() < need:
                raise ValueError(f"{nm} holds {t.numel() * t.element_size()} bytes, needs {need}")
    h = ctypes.c_void_p()
    c = cfg._c()
    _check(_lib.kv_cache_create(ctypes.byref(c), _dptr(k_pool, torch.float16, "k_pool"),
                                _dptr(v_pool, torch.float16, "v_pool"), ctypes.byref(h)), "kv_cache_create")
    _caches[h.value] = _Cache([] if k_pool is None else [k_pool, v_pool])
    return h.value


def kv_cache_destroy(h: int) -> None:
    cache = _caches.pop(getattr(h, "value", h), None)
    if cache is not None:
        cache.open = False
    _check(_lib.kv_cache_destroy(h), "kv_cache_destroy")


def kv_cache_layer(h: int, layer: int):
    k, v = ctypes.c_void_p(), ctypes.c_void_p()
    _check(_lib.kv_cache_layer(h, layer, ctypes.byref(k), ctypes.byref(v)), "kv_cache_layer")
    return k.value, v.value


def kv_block_alloc(h: int) -> int:
    b = ctypes.c_int32()
    _check(_lib.kv_block_alloc(h, ctypes.byref(b)), "kv_block_alloc")
    return b.value


def kv_block_share(h: int, block: int) -> None:
    _check(_lib.kv_block_share(h, int(block)), "kv_block_share")


def kv_block_release(h: int, block: int) -> None:
    _check(_lib.kv_block_release(h, int(block)), "kv_block_release")


def kv_block_refcount(h: int, block: int) -> int:
    r = ctypes.c_int32()
    _check(_lib.kv_block_refcount(h, int(block), ctypes.byref(r)), "kv_block_refcount")
    return r.value


def kv_block_num_free(h: int) -> int:
    r = ctypes.c_int32()
    _check(_lib.kv_block_num_free(h, ctypes.byref(r)), "kv_block_num_free")
    return r.value


def kv_cache_utilisation(h: int) -> float:
    r = ctypes.c_double()
    _check(_lib.kv_cache_utilisation(h, ctypes.byref(r)), "kv_cache_utilisation")
    return r.value


def kv_block_cow(h: int, block: int, stream=None) -> int:
    r = ctypes.c_int32()
    _check(_lib.kv_block_cow(h, int(block), ctypes.byref(r), _stream(stream)), "kv_block_cow")
    return r.value


def kv_copy_blocks(h: int, src: Sequence[int], dst: Sequence[int], stream=None) -> None:
    s, d = _host(src, np.int32), _host(dst, np.int32)
    if s.shape != d.shape:
        raise ValueError("src and dst differ in length")
    _check(_lib.kv_copy_blocks(h, _np_ptr(s), _np_ptr(d), len(s), _stream(stream)), "kv_copy_blocks")


# ------------------------------------------------------------ slots (host)
def kv_slot_mapping(block_table: np.ndarray, first_pos, count, block_size: int = 16) -> np.ndarray:
    table = _host(block_table, np.int32)
    fp, cn = _host(first_pos, np.int32), _host(count, np.int32)
    B, mb = table.shape
    out = np.empty(int(cn.astype(np.int64).sum()), dtype=np.int64)
    _check(_lib.kv_slot_mapping(_np_ptr(table), mb, B, _np_ptr(fp), _np_ptr(cn), block_size, _np_ptr(out)),
           "kv_slot_mapping")
    return out


def kv_step_prepare(h: int, block_table: np.ndarray, num_blocks: np.ndarray, positions):
    """One decode step's allocation / copy-on-write; block_table and num_blocks are updated in place.

    Returns (slot_mapping int64 [B], copy pairs int32 [n][2])."""
    if block_table.dtype != np.int32 or not block_table.flags.c_contiguous:
        raise TypeError("block_table must be a C-contiguous int32 array")
    if num_blocks.dtype != np.int32 or not num_blocks.flags.c_contiguous:
        raise TypeError("num_blocks must be a C-contiguous int32 array")
    pos = _host(positions, np.int32)
    B, mb = block_table.shape
    slots = np.empty(B, dtype=np.int64)
    src = np.empty(max(B, 1), dtype=np.int32)
    dst = np.empty(max(B, 1), dtype=np.int32)
    n = ctypes.c_int(0)
    _check(_lib.kv_step_prepare(h, _np_ptr(block_table), mb, _np_ptr(num_blocks), _np_ptr(pos), B, _np_ptr(slots),
                                _np_ptr(src), _np_ptr(dst), ctypes.byref(n)), "kv_step_prepare")
    return slots, np.stack([src[:n.value], dst[:n.value]], axis=1)


# ------------------------------------------------------------ device ops
def kv_append(h: int, layer: int, k_new: torch.Tensor, v_new: torch.Tensor, slot_mapping: torch.Tensor,
              stream=None, prepare: bool = False):
    """Scatter rows of k_new/v_new ([n][Hkv][D] fp16) to slot_mapping (int64 [n]) of one layer.

    prepare=True returns a PreparedCall instead of launching."""
    n = k_new.shape[0]
    if v_new.shape != k_new.shape or slot_mapping.numel() != n:
        raise ValueError("k_new, v_new and slot_mapping must agree in n")
    args = (h, layer, _dptr(k_new, torch.float16, "k_new"), _dptr(v_new, torch.float16, "v_new"),
            _dptr(slot_mapping, torch.int64, "slot_mapping"), n)
    return _launch(_lib.kv_append, args, "kv_append", stream, prepare, (k_new, v_new, slot_mapping))


def paged_decode_plan(B: int, Hq: int, Hkv: int, head_dim: int, max_context_len: int, blocks_per_split: int = 0,
                      block_size: int = 16):
    ns, bps, ws = ctypes.c_int(), ctypes.c_int(), ctypes.c_size_t()
    _check(_lib.paged_decode_plan(B, Hq, Hkv, head_dim, block_size, max_context_len, blocks_per_split,
                                  ctypes.byref(ns), ctypes.byref(bps), ctypes.byref(ws)), "paged_decode_plan")
    return ns.value, bps.value, ws.value


def paged_decode_workspace_init(workspace: torch.Tensor, stream=None) -> None:
    _check(_lib.paged_decode_workspace_init(_dptr(workspace, None, "workspace"),
                                            workspace.numel() * workspace.element_size(),
                                            _stream(stream, workspace)), "paged_decode_workspace_init")


def paged_decode_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                           context_lens: torch.Tensor, scale: float, out: torch.Tensor,
                           workspace: Optional[torch.Tensor], max_context_len: int, blocks_per_split: int = 0,
                           stream=None, prepare: bool = False):
    """out = softmax(q K^T * scale) V per sequence over its paged context.

    q [B][Hq][D] fp16; k_cache/v_cache [NB][Hkv][bs][D] fp16 (one layer); block_table int32 [B][max_blocks];
    context_lens int32 [B]; out [B][Hq][D] fp16 or fp32; workspace: paged_decode_plan(...) bytes (uint8/any).
    prepare=True returns a PreparedCall instead of launching.
    """
    B, Hq, D = q.shape
    NB, Hkv, bs, Dk = k_cache.shape
    if Dk != D or v_cache.shape != k_cache.shape:
        raise ValueError("cache shapes do not match q")
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    if block_table.dim() != 2 or block_table.shape[0] != B or context_lens.numel() != B:
        raise ValueError("block_table / context_lens do not match B")
    if out.dtype == torch.float16:
        od = KVC_F16
    elif out.dtype == torch.float32:
        od = KVC_F32
    else:
        raise TypeError("out must be float16 or float32")
    ws_ptr = _dptr(workspace, None, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    args = (_dptr(q, torch.float16, "q"), _dptr(k_cache, torch.float16, "k_cache"),
            _dptr(v_cache, torch.float16, "v_cache"), NB, _dptr(block_table, torch.int32, "block_table"),
            block_table.shape[1], _dptr(context_lens, torch.int32, "context_lens"), B, Hq, Hkv, D, bs,
            int(max_context_len), float(scale), _dptr(out, None, "out"), od, ws_ptr, ws_bytes,
            int(blocks_per_split))
    return _launch(_lib.paged_decode_attention, args, "paged_decode_attention", stream, prepare,
                   (q, k_cache, v_cache, block_table, context_lens, out, workspace))


def kv_cascade_groups(block_table: np.ndarray, context_lens, max_group: int = 8, block_size: int = 16):
    """Groups for paged_decode_cascade_attention from a host block table [B][max_blocks] and context lengths:
    returns (group_start int32 [n_groups + 1], shared_blocks int32 [B], max_shared)."""
    table = _host(block_table, np.int32)
    if table.ndim != 2:
        raise ValueError("block_table must be [B][max_blocks]")
    B, mb = table.shape
    ctx = _host(context_lens, np.int32)
    gs = np.zeros(B + 1, dtype=np.int32)
    sh = np.zeros(max(B, 1), dtype=np.int32)
    ng, mx = ctypes.c_int(), ctypes.c_int()
    _check(_lib.kv_cascade_groups(_np_ptr(table), B, mb, _np_ptr(ctx), block_size, max_group, _np_ptr(gs),
                                  ctypes.byref(ng), _np_ptr(sh), ctypes.byref(mx)), "kv_cascade_groups")
    return gs[:ng.value + 1].copy(), sh[:B].copy(), mx.value


def paged_decode_cascade_plan(B: int, Hq: int, Hkv: int, head_dim: int, max_context_len: int, n_groups: int,
                              max_shared_blocks: int, block_size: int = 16) -> int:
    """Workspace bytes of paged_decode_cascade_attention for these sizes."""
    ws = ctypes.c_size_t()
    _check(_lib.paged_decode_cascade_plan(B, Hq, Hkv, head_dim, block_size, max_context_len, n_groups,
                                          max_shared_blocks, ctypes.byref(ws)), "paged_decode_cascade_plan")
    return ws.value


def paged_decode_cascade_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                   block_table: torch.Tensor, context_lens: torch.Tensor, group_start: torch.Tensor,
                                   shared_blocks: torch.Tensor, max_shared_blocks: int, scale: float,
                                   out: torch.Tensor, workspace: torch.Tensor, max_context_len: int,
                                   stream=None) -> None:
    """paged_decode_attention's result, with each group's shared leading blocks read once for the group.

    group_start int32 [n_groups + 1] (groups of consecutive sequences, at most 8 each); shared_blocks int32 [B]
    (leading blocks every member of the sequence's group has in common); workspace: paged_decode_cascade_plan bytes.
    """
    B, Hq, D = q.shape
    NB, Hkv, bs, Dk = k_cache.shape
    if Dk != D or v_cache.shape != k_cache.shape:
        raise ValueError("cache shapes do not match q")
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    if block_table.dim() != 2 or block_table.shape[0] != B or context_lens.numel() != B:
        raise ValueError("block_table / context_lens do not match B")
    if shared_blocks.numel() != B or group_start.numel() < 2:
        raise ValueError("shared_blocks must have B entries and group_start at least 2")
    if out.dtype == torch.float16:
        od = KVC_F16
    elif out.dtype == torch.float32:
        od = KVC_F32
    else:
        raise TypeError("out must be float16 or float32")
    _check(_lib.paged_decode_cascade_attention(
        _dptr(q, torch.float16, "q"), _dptr(k_cache, torch.float16, "k_cache"),
        _dptr(v_cache, torch.float16, "v_cache"), NB, _dptr(block_table, torch.int32, "block_table"),
        block_table.shape[1], _dptr(context_lens, torch.int32, "context_lens"),
        _dptr(group_start, torch.int32, "group_start"), _dptr(shared_blocks, torch.int32, "shared_blocks"),
        group_start.numel() - 1, int(max_shared_blocks), B, Hq, Hkv, D, bs, int(max_context_len), float(scale),
        _dptr(out, None, "out"), od, _dptr(workspace, None, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream, q)), "paged_decode_cascade_attention")


def paged_decode_multi_plan(B: int, Hq: int, Hkv: int, head_dim: int, max_context_len: int, q_len: int,
                            block_size: int = 16) -> int:
    """Workspace bytes of paged_decode_multi_attention for these sizes."""
    ws = ctypes.c_size_t()
    _check(_lib.paged_decode_multi_plan(B, Hq, Hkv, head_dim, block_size, max_context_len, q_len, ctypes.byref(ws)),
           "paged_decode_multi_plan")
    return ws.value


def paged_decode_multi_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                 block_table: torch.Tensor, context_lens: torch.Tensor, scale: float,
                                 out: torch.Tensor, workspace: torch.Tensor, max_context_len: int,
                                 stream=None) -> None:
    """q [B][q_len][Hq][D] fp16: the q_len newest tokens of every sequence (already in the cache), causal among
    themselves; out like q (fp16 or fp32); workspace: paged_decode_multi_plan bytes."""
    B, T, Hq, D = q.shape
    NB, Hkv, bs, Dk = k_cache.shape
    if Dk != D or v_cache.shape != k_cache.shape:
        raise ValueError("cache shapes do not match q")
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    if block_table.dim() != 2 or block_table.shape[0] != B or context_lens.numel() != B:
        raise ValueError("block_table / context_lens do not match B")
    if out.dtype == torch.float16:
        od = KVC_F16
    elif out.dtype == torch.float32:
        od = KVC_F32
    else:
        raise TypeError("out must be float16 or float32")
    _check(_lib.paged_decode_multi_attention(
        _dptr(q, torch.float16, "q"), _dptr(k_cache, torch.float16, "k_cache"),
        _dptr(v_cache, torch.float16, "v_cache"), NB, _dptr(block_table, torch.int32, "block_table"),
        block_table.shape[1], _dptr(context_lens, torch.int32, "context_lens"), T, B, Hq, Hkv, D, bs,
        int(max_context_len), float(scale), _dptr(out, None, "out"), od, _dptr(workspace, None, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream, q)), "paged_decode_multi_attention")


def fp8_v_position(tau: int) -> int:
    """Byte position of token tau (0..15) of a block within each 16-byte dim row of an fp8 record's V codes."""
    return 4 * ((tau & 7) >> 1) + 2 * (tau >> 3) + (tau & 1)


def kv_fp8_record_bytes(head_dim: int) -> int:
    """Bytes of one fp8 cache record (one per (block, KV head)): 32 * head_dim + 128."""
    n = ctypes.c_size_t()
    _check(_lib.kv_fp8_record_bytes(int(head_dim), ctypes.byref(n)), "kv_fp8_record_bytes")
    return n.value


def kv_append_fp8(k_new: torch.Tensor, v_new: torch.Tensor, slot_mapping: torch.Tensor, kv_fp8: torch.Tensor,
                  stream=None) -> None:
    """Quantize k_new / v_new (fp16 [n][Hkv][D]) into an fp8 cache layer kv_fp8, uint8 [NB][Hkv][record] (one
    record of kv_fp8_record_bytes(D) per (block, KV head): K codes, K scales, V codes, V scales; value = e4m3
    code value * scale); slot_mapping int64 [n]."""
    n, Hkv, D = k_new.shape
    NB, Hkv2, rec = kv_fp8.shape
    if Hkv2 != Hkv or rec != kv_fp8_record_bytes(D) or v_new.shape != k_new.shape or slot_mapping.numel() != n:
        raise ValueError("fp8 cache shapes do not match")
    _check(_lib.kv_append_fp8(
        _dptr(k_new, torch.float16, "k_new"), _dptr(v_new, torch.float16, "v_new"),
        _dptr(slot_mapping, torch.int64, "slot_mapping"), n, _dptr(kv_fp8, torch.uint8, "kv_fp8"), NB, Hkv, D, 16,
        _stream(stream, k_new)), "kv_append_fp8")


def paged_decode_attention_fp8(q: torch.Tensor, kv_fp8: torch.Tensor, block_table: torch.Tensor,
                               context_lens: torch.Tensor, scale: float, out: torch.Tensor,
                               workspace: Optional[torch.Tensor], max_context_len: int, blocks_per_split: int = 0,
                               stream=None) -> None:
    """paged_decode_attention over an fp8 cache layer (kv_fp8 uint8 [NB][Hkv][record] as kv_append_fp8 writes it)."""
    B, Hq, D = q.shape
    NB, Hkv, rec = kv_fp8.shape
    if rec != kv_fp8_record_bytes(D):
        raise ValueError("fp8 cache records do not match q's head dim")
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    if block_table.dim() != 2 or block_table.shape[0] != B or context_lens.numel() != B:
        raise ValueError("block_table / context_lens do not match B")
    od = {torch.float16: KVC_F16, torch.float32: KVC_F32}.get(out.dtype)
    if od is None:
        raise TypeError("out must be float16 or float32")
    ws_ptr = _dptr(workspace, None, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(_lib.paged_decode_attention_fp8(
        _dptr(q, torch.float16, "q"), _dptr(kv_fp8, torch.uint8, "kv_fp8"), NB,
        _dptr(block_table, torch.int32, "block_table"), block_table.shape[1],
        _dptr(context_lens, torch.int32, "context_lens"), B, Hq, Hkv, D, 16, int(max_context_len), float(scale),
        _dptr(out, None, "out"), od, ws_ptr, ws_bytes, int(blocks_per_split), _stream(stream, q)),
        "paged_decode_attention_fp8")


def paged_decode_append_attention(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, k_cache: torch.Tensor,
                                  v_cache: torch.Tensor, block_table: torch.Tensor, context_lens: torch.Tensor,
                                  scale: float, out: torch.Tensor, workspace: Optional[torch.Tensor],
                                  max_context_len: int, blocks_per_split: int = 0, stream=None,
                                  prepare: bool = False):
    """Append k_new/v_new ([B][Hkv][D] fp16) at position ctx-1 of every sequence, then attend (one kernel).

    prepare=True returns a PreparedCall instead of launching."""
    B, Hq, D = q.shape
    NB, Hkv, bs, Dk = k_cache.shape
    if Dk != D or v_cache.shape != k_cache.shape or out.shape != q.shape:
        raise ValueError("shape mismatch")
    if k_new.shape != (B, Hkv, D) or v_new.shape != k_new.shape:
        raise ValueError("k_new/v_new must be [B][Hkv][D]")
    if block_table.dim() != 2 or block_table.shape[0] != B or context_lens.numel() != B:
        raise ValueError("block_table / context_lens do not match B")
    od = KVC_F16 if out.dtype == torch.float16 else KVC_F32 if out.dtype == torch.float32 else None
    if od is None:
        raise TypeError("out must be float16 or float32")
    ws_ptr = _dptr(workspace, None, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    args = (_dptr(q, torch.float16, "q"), _dptr(k_new, torch.float16, "k_new"), _dptr(v_new, torch.float16, "v_new"),
            _dptr(k_cache, torch.float16, "k_cache"), _dptr(v_cache, torch.float16, "v_cache"), NB,
            _dptr(block_table, torch.int32, "block_table"), block_table.shape[1],
            _dptr(context_lens, torch.int32, "context_lens"), B, Hq, Hkv, D, bs, int(max_context_len), float(scale),
            _dptr(out, None, "out"), od, ws_ptr, ws_bytes, int(blocks_per_split))
    return _launch(_lib.paged_decode_append_attention, args, "paged_decode_append_attention", stream, prepare,
                   (q, k_new, v_new, k_cache, v_cache, block_table, context_lens, out, workspace))


def paged_decode_attention_static_workspace(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                            block_table: torch.Tensor, context_lens: torch.Tensor, scale: float,
                                            out: torch.Tensor, max_context_len: int, blocks_per_split: int = 0,
                                            stream=None) -> None:
    """paged_decode_attention without a workspace argument: split scratch comes from the library's fixed
    16 MiB device array, so the call allocates nothing (for callers that must not allocate device memory).

    The first call on a device looks up that array's address; make it before any stream capture. Calls that
    overlap on the GPU share the array and race on it."""
    B, Hq, D = q.shape
    NB, Hkv, bs, Dk = k_cache.shape
    if Dk != D or v_cache.shape != k_cache.shape or out.shape != q.shape:
        raise ValueError("shape mismatch")
    if block_table.dim() != 2 or block_table.shape[0] != B or context_lens.numel() != B:
        raise ValueError("block_table / context_lens do not match B")
    od = KVC_F16 if out.dtype == torch.float16 else KVC_F32 if out.dtype == torch.float32 else None
    if od is None:
        raise TypeError("out must be float16 or float32")
    _check(_lib.paged_decode_attention_static_workspace(
        _dptr(q, torch.float16, "q"), _dptr(k_cache, torch.float16, "k_cache"),
        _dptr(v_cache, torch.float16, "v_cache"), NB, _dptr(block_table, torch.int32, "block_table"),
        block_table.shape[1], _dptr(context_lens, torch.int32, "context_lens"), B, Hq, Hkv, D, bs,
        int(max_context_len), float(scale), _dptr(out, None, "out"), od, int(blocks_per_split), _stream(stream, q)),
        "paged_decode_attention_static_workspace")


def paged_decode_attention_raw(q_ptr: int, k_ptr: int, v_ptr: int, num_blocks: int, table_ptr: int, max_blocks: int,
                               ctx_ptr: int, B: int, Hq: int, Hkv: int, D: int, max_context_len: int, scale: float,
                               out_ptr: int, out_dtype: int, ws_ptr: int, ws_bytes: int, blocks_per_split: int,
                               stream: int) -> None:
    """Same call with raw device pointers (e.g. a layer slice from kv_cache_layer)."""
    _check(_lib.paged_decode_attention(q_ptr, k_ptr, v_ptr, num_blocks, table_ptr, max_blocks, ctx_ptr, B, Hq, Hkv,
                                       D, 16, max_context_len, float(scale), out_ptr, out_dtype, ws_ptr, ws_bytes,
                                       blocks_per_split, stream), "paged_decode_attention")


def prefill_attention_ex(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                         max_seqlen: int, scale: float, causal: bool, p_precision: int, out: torch.Tensor,
                         stream=None) -> None:
    """Packed varlen prefill with a choice of P precision (KVC_PREFILL_P_F16 or KVC_PREFILL_P_SPLIT):
    q [T][Hq][D], k/v [T][Hkv][D] fp16, cu_seqlens int32 [nseq+1] -> out [T][Hq][D]."""
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    if k.shape != (T, Hkv, D) or v.shape != k.shape or out.shape != q.shape:
        raise ValueError("shape mismatch")
    od = KVC_F16 if out.dtype == torch.float16 else KVC_F32 if out.dtype == torch.float32 else None
    if od is None:
        raise TypeError("out must be float16 or float32")
    _check(_lib.prefill_attention_ex(_dptr(q, torch.float16, "q"), _dptr(k, torch.float16, "k"),
                                     _dptr(v, torch.float16, "v"), _dptr(cu_seqlens, torch.int32, "cu_seqlens"),
                                     cu_seqlens.numel() - 1, T, int(max_seqlen), Hq, Hkv, D, float(scale),
                                     int(bool(causal)), int(p_precision), _dptr(out, None, "out"), od,
                                     _stream(stream, q)),
           "prefill_attention_ex")


def prefill_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, max_seqlen: int,
                      scale: float, causal: bool, out: torch.Tensor, stream=None, precise: bool = False) -> None:
    """Packed varlen prefill: q [T][Hq][D], k/v [T][Hkv][D] fp16, cu_seqlens int32 [nseq+1] -> out [T][Hq][D].

    precise=False rounds the softmax weights P to fp16 (KVC_PREFILL_P_F16); precise=True multiplies V by
    P's fp16 high part and residual (KVC_PREFILL_P_SPLIT)."""
    prefill_attention_ex(q, k, v, cu_seqlens, max_seqlen, scale, causal,
                         KVC_PREFILL_P_SPLIT if precise else KVC_PREFILL_P_F16, out, stream)


# ------------------------------------------------------------ tree-drafted decoding
def kv_tree_masks(parents, tree_lens=None):
    """Masks (int64 [B][T], the bits of a node and its ancestors) and depths (int32 [B][T]) of drafted trees from
    their parents [B][T] (host arrays; a node's parent has a smaller index, node 0 is the root)."""
    par = _host(parents, np.int32)
    if par.ndim != 2:
        raise ValueError("parents must be [B][T]")
    B, T = par.shape
    lens = None if tree_lens is None else _host(tree_lens, np.int32)
    if lens is not None and lens.shape != (B,):
        raise ValueError("tree_lens must have B entries")
    masks, depths = np.zeros((B, T), np.int64), np.zeros((B, T), np.int32)
    _check(_lib.kv_tree_masks(_np_ptr(par), None if lens is None else _np_ptr(lens), B, T, _np_ptr(masks),
                              _np_ptr(depths)), "kv_tree_masks")
    return masks, depths


def kv_rope_turns(inv_freq) -> np.ndarray:
    """Rotation frequencies (radians per position, one per pair) as fractions of a turn in units of 2^-64: the int64
    bit patterns kv_append_rope takes (copy them to the device)."""
    f = _host(inv_freq, np.float64)
    if f.ndim != 1:
        raise ValueError("inv_freq must be one-dimensional")
    turns = np.zeros(f.size, np.int64)
    _check(_lib.kv_rope_turns(_np_ptr(f), f.size, _np_ptr(turns)), "kv_rope_turns")
    return turns


_F16, _F32, _I32, _I64 = torch.float16, torch.float32, torch.int32, torch.int64
_U8, _E4M3 = torch.uint8, torch.float8_e4m3fn
# the current device's index (the underscored form skips a wrapper, 0.1 µs a call)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _same_device(*tensors) -> None:
    """Every tensor given (None: left out) is on the current device, where the library's kernels run."""
    devices = {t.device for t in tensors if t is not None}
    if len(devices) > 1:
        raise ValueError("tensors are on several devices: " + ", ".join(sorted(map(str, devices))))
    for d in devices:
        if d.type == "cuda" and d.index != _current_device():
            raise ValueError(f"tensors are on {d}, the current device is cuda:{_current_device()}")


def _ready(dev: int, dtype, *tensors) -> bool:
    """Every tensor given (None: left out) is a contiguous CUDA tensor of the type on device dev: the test of a call's
    common case in one go.  Where it fails, the call's own checks name what is wrong."""
    for t in tensors:
        if t is not None and (t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous()):
            return False
    return True


class _Words:
    """A launching call of kvc_call: its number and its arguments' places in the array of words."""
    __slots__ = ("which", "count", "pack", "name")

    def __init__(self, which: int, name: str):
        types = getattr(_lib, name).argtypes[:-1]  # without the stream
        self.which, self.count, self.name = which, len(types), name
        self.pack = struct.Struct("=" + "".join("d" if t is ctypes.c_float else "q" for t in types)).pack


_APPEND_ROPE, _TREE_ATTENTION, _TREE_VERIFY, _TREE_COMMIT = (
    _Words(i + 1, name) for i, name in enumerate(("kv_append_rope", "paged_decode_tree_attention", "draft_tree_verify",
                                                  "kv_tree_commit")))
_BLOCK_TABLES, _APPEND_FP8_BLOCK, _ATTENTION_FP8_BLOCK, _WINDOW_ATTENTION, _PREFILL_WINDOW = (
    _Words(i + 16, name) for i, name in enumerate((
        "kv_block_tables", "kv_append_fp8_block", "paged_decode_attention_fp8_block", "paged_decode_window_attention",
        "prefill_window_attention")))
_call = _lib.kvc_call


def _run(call: _Words, args, stream, prepare, dev, keep, cache=None):
    """Launch the call with args (0 for a null pointer) on `stream` or the current one of device dev, or return it as a
    PreparedCall.  The arguments go as one array: ctypes takes ~60 ns for each of up to 26."""
    words = call.pack(*args)
    if prepare and cache is not None:
        return _PreparedCacheCall(_call, (call.which, words, call.count), call.name, dev, keep, cache)
    if prepare:
        return PreparedCall(_call, (call.which, words, call.count), call.name, dev, keep)
    if stream is None and _raw_stream is not None:
        st = _raw_stream(dev)
    else:
        st = _stream(stream, keep[0])
    status = _call(call.which, words, call.count, st)
    if status:
        _check(status, call.name)
    return None


def kvc_call(which: int, words: bytes, stream=None) -> None:
    """A launching call by its number (KVC_CALL_* of the header) with its arguments as 64-bit words, on `stream` or the
    current one: the library's call as it is, for bindings of one's own.  Addresses are not checked (a wrong one is a
    fault on the device), nor is what they belong to kept alive; the calls' own functions build the words from
    tensors, check those and keep them."""
    if len(words) % 8:
        raise ValueError("words must be whole 64-bit words")
    st = torch.cuda.current_stream().cuda_stream if stream is None and torch.cuda.is_available() else _stream(stream)
    _check(_call(which, words, len(words) // 8, st), "kvc_call")


def _token_stride(t: torch.Tensor, name: str) -> int:
    """Token stride of an [n][H][D] fp16 tensor whose heads are packed and whose tokens may be apart."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if t.dtype != torch.float16:
        raise TypeError(f"{name} must be torch.float16, got {t.dtype}")
    n, H, D = t.shape
    if (D > 1 and t.stride(2) != 1) or (H > 1 and t.stride(1) != D):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    return t.stride(0) if n > 1 else H * D


def kv_append_rope(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: Optional[torch.Tensor],
                   turns: Optional[torch.Tensor], q_out: torch.Tensor, k_cache: Optional[torch.Tensor] = None,
                   v_cache: Optional[torch.Tensor] = None, slot_mapping: Optional[torch.Tensor] = None, *,
                   q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                   eps: float = 1e-6, interleaved: bool = False, k_out: Optional[torch.Tensor] = None,
                   v_out: Optional[torch.Tensor] = None, stream=None, prepare: bool = False):
    """Norm and rotate query and key rows and append keys and values to the paged cache, in one pass.

    q [n][Hq][D], k and v [n][Hkv][D] fp16 (the tokens may be apart, as parts of one projection's output); positions
    int32 [n]; turns int64 [rot_dim / 2] (kv_rope_turns; None: no rotation); q_out [n][Hq][D]; k_cache / v_cache
    [NB][Hkv][bs][D] (one layer) with slot_mapping int64 [n]; q_weight / k_weight fp16 [D] (None: no norm);
    k_out / v_out [n][Hkv][D]: the rows packed.  prepare=True returns a PreparedCall instead of launching."""
    qshape, kshape, rot, NB, bs = q.shape, k.shape, 0, 0, 16
    if len(qshape) != 3 or len(kshape) != 3:
        raise ValueError("q, k and v must be [n][H][D]")
    n, Hq, D = qshape
    kn, Hkv, kd = kshape
    if kn != n or kd != D or v.shape != kshape or q_out.shape != qshape:
        raise ValueError("q, k, v and q_out do not match")
    if turns is not None and (half := turns.numel()):
        rot = 2 * half
        if positions is None or positions.numel() != n:
            raise ValueError("positions must have n entries")
    else:
        positions = turns = None
    if k_cache is not None and v_cache is not None and slot_mapping is not None:
        cshape = k_cache.shape
        if len(cshape) != 4:
            raise ValueError("k_cache must be [NB][Hkv][bs][D]")
        NB, Hc, bs, Dc = cshape
        if Hc != Hkv or Dc != D or v_cache.shape != cshape:
            raise ValueError("cache shapes do not match k")
        if slot_mapping.numel() != n:
            raise ValueError("slot_mapping must have n entries")
    elif k_cache is not None or v_cache is not None or slot_mapping is not None:
        raise ValueError("k_cache, v_cache and slot_mapping: all or none")
    if (q_weight is not None and q_weight.numel() != D) or (k_weight is not None and k_weight.numel() != D):
        raise ValueError("q_weight and k_weight must have D entries")
    if (k_out is not None and k_out.shape != kshape) or (v_out is not None and v_out.shape != kshape):
        raise ValueError("k_out and v_out must have k's shape")
    keep = (q, k, v, positions, turns, q_out, k_cache, v_cache, slot_mapping, q_weight, k_weight, k_out, v_out)
    dev = q.get_device()
    qst, kst, vst = q.stride(), k.stride(), v.stride()
    # the common case in one expression; the checks below only name the failure
    if not (dev >= 0 and dev == _current_device() == k.get_device() == v.get_device()
            and q.dtype is _F16 and k.dtype is _F16 and v.dtype is _F16
            and qst[2] == kst[2] == vst[2] == 1 and qst[1] == kst[1] == vst[1] == D
            and _ready(dev, _F16, q_out, q_weight, k_weight, k_out, v_out, k_cache, v_cache)
            and _ready(dev, _I64, turns, slot_mapping) and _ready(dev, _I32, positions)):
        qst, kst, vst = ((_token_stride(t, nm),) for t, nm in ((q, "q"), (k, "k"), (v, "v")))
        _same_device(*keep)
        for t, nm in ((q_weight, "q_weight"), (k_weight, "k_weight"), (q_out, "q_out"), (k_out, "k_out"),
                      (v_out, "v_out"), (k_cache, "k_cache"), (v_cache, "v_cache")):
            _dptr(t, _F16, nm)
        for t, nm in ((turns, "turns"), (slot_mapping, "slot_mapping")):
            _dptr(t, _I64, nm)
        _dptr(positions, _I32, "positions")
    if n == 1:  # a single token's stride means nothing
        qst, kst, vst = (Hq * D,), (Hkv * D,), (Hkv * D,)
    args = (q.data_ptr(), qst[0], k.data_ptr(), kst[0], v.data_ptr(), vst[0], n, Hq, Hkv, D,
            0 if q_weight is None else q_weight.data_ptr(),
            0 if k_weight is None else k_weight.data_ptr(), float(eps), 0 if turns is None else turns.data_ptr(), rot,
            1 if interleaved else 0, 0 if positions is None else positions.data_ptr(), q_out.data_ptr(),
            0 if k_out is None else k_out.data_ptr(), 0 if v_out is None else v_out.data_ptr(),
            0 if k_cache is None else k_cache.data_ptr(), 0 if v_cache is None else v_cache.data_ptr(), NB, bs,
            0 if slot_mapping is None else slot_mapping.data_ptr())
    return _run(_APPEND_ROPE, args, stream, prepare, dev, keep)


def paged_decode_tree_plan(B: int, Hq: int, Hkv: int, head_dim: int, max_context_len: int, T: int,
                           block_size: int = 16) -> int:
    """Workspace bytes of paged_decode_tree_attention for these sizes (trees of up to T nodes)."""
    ws = ctypes.c_size_t()
    _check(_lib.paged_decode_tree_plan(B, Hq, Hkv, head_dim, block_size, max_context_len, T, ctypes.byref(ws)),
           "paged_decode_tree_plan")
    return ws.value


def paged_decode_tree_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                block_table: torch.Tensor, context_lens: torch.Tensor, masks: torch.Tensor,
                                scale: float, out: torch.Tensor, workspace: Optional[torch.Tensor],
                                max_context_len: int, tree_lens: Optional[torch.Tensor] = None, stream=None,
                                prepare: bool = False):
    """Attention of drafted trees (the newest tree_lens[b] cached tokens of every sequence) over the paged cache.

    q [B][T][Hq][D] fp16; masks int64 [B][T] (kv_tree_masks: bit j of a row = it sees node j; every row sees the
    history); context_lens int32 [B], trees included; tree_lens int32 [B] (None: T nodes each; rows behind a tree are
    left as they were); out like q, fp16 or fp32; workspace: paged_decode_tree_plan bytes.
    prepare=True returns a PreparedCall instead of launching."""
    qshape = q.shape
    B, T, Hq, D = qshape
    NB, Hkv, bs, Dk = k_cache.shape
    if Dk != D or v_cache.shape != k_cache.shape:
        raise ValueError("cache shapes do not match q")
    if out.shape != qshape:
        raise ValueError("out must have q's shape")
    if block_table.dim() != 2 or block_table.shape[0] != B or context_lens.numel() != B:
        raise ValueError("block_table / context_lens do not match B")
    if masks.shape != (B, T) or (tree_lens is not None and tree_lens.numel() != B):
        raise ValueError("masks must be [B][T] and tree_lens have B entries")
    odt = out.dtype
    od = KVC_F16 if odt is _F16 else KVC_F32 if odt is _F32 else None
    if od is None:
        raise TypeError("out must be float16 or float32")
    keep = (q, k_cache, v_cache, block_table, context_lens, masks, tree_lens, out, workspace)
    dev = q.get_device()
    if not (dev >= 0 and dev == _current_device() and _ready(dev, _F16, q, k_cache, v_cache, out if od == KVC_F16 else None)
            and _ready(dev, _I32, block_table, context_lens, tree_lens) and masks.dtype is _I64
            and masks.get_device() == dev and masks.is_contiguous() and (od == KVC_F16 or _ready(dev, _F32, out))
            and (workspace is None or _ready(dev, workspace.dtype, workspace))):
        _same_device(*keep)
        for t, dt, nm in ((q, _F16, "q"), (k_cache, _F16, "k_cache"), (v_cache, _F16, "v_cache"),
                          (block_table, _I32, "block_table"), (context_lens, _I32, "context_lens"),
                          (masks, _I64, "masks"), (tree_lens, _I32, "tree_lens"), (out, None, "out"),
                          (workspace, None, "workspace")):
            _dptr(t, dt, nm)
    args = (q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), NB, block_table.data_ptr(), block_table.shape[1],
            context_lens.data_ptr(), masks.data_ptr(), 0 if tree_lens is None else tree_lens.data_ptr(), T, B, Hq,
            Hkv, D, bs, int(max_context_len), float(scale), out.data_ptr(), od,
            0 if workspace is None else workspace.data_ptr(),
            0 if workspace is None else workspace.numel() * workspace.element_size())
    return _run(_TREE_ATTENTION, args, stream, prepare, dev, keep)


def _prob_rows(t: torch.Tensor, name: str):
    """Pointer and row stride of a [B][T][V] tensor with contiguous rows at one distance from each other."""
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in (torch.float32, torch.float16) and t.dim() == 3 \
            and t.is_contiguous():
        return t.data_ptr(), t.shape[2]  # the common case; the checks below name the failure
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [B][T][V]")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if t.dtype not in (torch.float16, torch.float32):
        raise TypeError(f"{name} must be float16 or float32")
    B, T, V = t.shape
    row = t.stride(1) if T > 1 else t.stride(0) if B > 1 else V
    if (V > 1 and t.stride(2) != 1) or (B > 1 and T > 1 and t.stride(0) != T * row):
        raise ValueError(f"{name}: rows must be contiguous and evenly spaced")
    return t.data_ptr(), row


def draft_tree_verify(target_probs: torch.Tensor, draft_probs: torch.Tensor, tokens: torch.Tensor,
                      parents: torch.Tensor, uniforms: torch.Tensor, path: torch.Tensor, path_len: torch.Tensor,
                      next_token: torch.Tensor, tree_lens: Optional[torch.Tensor] = None, distinct: bool = False,
                      stream=None, prepare: bool = False):
    """Which drafted tokens the target keeps (path int32 [B][T]: the kept nodes, root first, then -1; path_len int32
    [B]) and the token after them (next_token int32 [B]).

    target_probs / draft_probs [B][T][V] fp32 or fp16 (row t: the distribution behind node t); tokens / parents int32
    [B][T]; uniforms fp32 [B][T] in [0, 1) (entry 0 draws the next token); tree_lens int32 [B] (None: T nodes each);
    distinct: a node's children were drawn without replacement.  prepare=True returns a PreparedCall."""
    pp, ps = _prob_rows(target_probs, "target_probs")
    qp, qs = _prob_rows(draft_probs, "draft_probs")
    shape, pdt = target_probs.shape, target_probs.dtype
    B, T, V = shape
    if draft_probs.shape != shape or draft_probs.dtype is not pdt:
        raise ValueError("target_probs and draft_probs must agree in shape and type")
    rows = tokens.shape
    if rows != (B, T) or parents.shape != rows or uniforms.shape != rows or path.shape != rows:
        raise ValueError("tokens, parents, uniforms and path must be [B][T]")
    if path_len.numel() != B or next_token.numel() != B or (tree_lens is not None and tree_lens.numel() != B):
        raise ValueError("path_len, next_token and tree_lens must have B entries")
    keep = (target_probs, draft_probs, tokens, parents, tree_lens, uniforms, path, path_len, next_token)
    dev = target_probs.get_device()
    if not (dev >= 0 and dev == _current_device() == draft_probs.get_device()
            and _ready(dev, _I32, tokens, parents, path, path_len, next_token, tree_lens)
            and uniforms.dtype is _F32 and uniforms.get_device() == dev and uniforms.is_contiguous()):
        _same_device(*keep)
        for t, nm in ((tokens, "tokens"), (parents, "parents"), (tree_lens, "tree_lens"), (path, "path"),
                      (path_len, "path_len"), (next_token, "next_token")):
            _dptr(t, _I32, nm)
        _dptr(uniforms, _F32, "uniforms")
    args = (pp, ps, qp, qs, KVC_F32 if pdt is _F32 else KVC_F16, tokens.data_ptr(), parents.data_ptr(),
            0 if tree_lens is None else tree_lens.data_ptr(), uniforms.data_ptr(), B, T, V, 1 if distinct else 0,
            path.data_ptr(), path_len.data_ptr(), next_token.data_ptr())
    return _run(_TREE_VERIFY, args, stream, prepare, dev, keep)


def kv_tree_commit(h: int, block_table: torch.Tensor, context_lens: torch.Tensor, path: torch.Tensor,
                   path_len: torch.Tensor, new_context_lens: torch.Tensor, tree_lens: Optional[torch.Tensor] = None,
                   stream=None, prepare: bool = False):
    """Move the kept nodes' cache rows (path int32 [B][P], path_len int32 [B]; all layers of the handle's pools) to
    the end of their contexts and write the new context lengths (int32 [B], not context_lens itself).

    block_table int32 [B][max_blocks] and context_lens int32 [B] (trees included) as the attention call had them;
    tree_lens int32 [B] (None: P nodes each).  prepare=True returns a PreparedCall, which also keeps the pools alive and
    raises ValueError once the cache is destroyed."""
    cache = _open_cache(h)
    if path.dim() != 2 or block_table.dim() != 2:
        raise ValueError("path must be [B][P] and block_table [B][max_blocks]")
    B, P = path.shape
    nb, max_blocks = block_table.shape
    if nb != B:
        raise ValueError("block_table does not match path")
    if context_lens.numel() != B or path_len.numel() != B or new_context_lens.numel() != B or (
            tree_lens is not None and tree_lens.numel() != B):
        raise ValueError("context_lens, path_len, new_context_lens and tree_lens must have B entries")
    keep = (path, block_table, context_lens, tree_lens, path_len, new_context_lens)
    dev = path.get_device()
    if not (dev >= 0 and dev == _current_device()
            and _ready(dev, _I32, path, block_table, context_lens, path_len, new_context_lens, tree_lens)):
        _same_device(*keep)
        for t, nm in ((path, "path"), (block_table, "block_table"), (context_lens, "context_lens"),
                      (tree_lens, "tree_lens"), (path_len, "path_len"), (new_context_lens, "new_context_lens")):
            _dptr(t, _I32, nm)
    if cache.device is not None and cache.device != dev:
        raise ValueError(f"the tensors are on cuda:{dev}, the cache's pools on cuda:{cache.device}")
    args = (h, block_table.data_ptr(), max_blocks, context_lens.data_ptr(),
            0 if tree_lens is None else tree_lens.data_ptr(), path.data_ptr(), path_len.data_ptr(), P, B,
            new_context_lens.data_ptr())
    return _run(_TREE_COMMIT, args, stream, prepare, dev, keep, cache)


# ------------------------------------------------------------ windows, the block-scaled cache, tables built on the GPU
def _check_all(keep, *named) -> None:
    """The checks of a call whose common case failed: they name what is wrong.  named: (tensor or None, type, name)."""
    for t, _, nm in named:
        if t is not None and not isinstance(t, torch.Tensor):
            raise TypeError(f"{nm} must be a torch.Tensor")
    _same_device(*keep)
    for t, dt, nm in named:
        _dptr(t, dt, nm)


def kv_block_tables(lens_before: Optional[torch.Tensor], lens_after: torch.Tensor, free_blocks: torch.Tensor,
                    placed: torch.Tensor, block_table: torch.Tensor, new_placed: torch.Tensor, cu_tokens: torch.Tensor,
                    slot_mapping: torch.Tensor, positions: Optional[torch.Tensor] = None, window: int = 0,
                    sinks: int = 0, block_size: int = 16, stream=None, prepare: bool = False):
    """Block tables, slots and positions of one step, built on the GPU from the request lengths.

    lens_before (None: prompts, 0 each) / lens_after int32 [B]; free_blocks int32: blocks claimed from the pool, of which
    placed (int32 [1]) are used already; block_table int32 [B][max_blocks], the new blocks' entries written; new_placed
    int32 [1]; cu_tokens int32 [B + 1]; slot_mapping int64 [num_slots], -1 behind the last token; positions int32
    [num_slots].  With a window (and sinks) a sequence's blocks are used in turn, see include/kvc.h.
    prepare=True returns a PreparedCall instead of launching."""
    tshape = block_table.shape
    if len(tshape) != 2:
        raise ValueError("block_table must be [B][max_blocks]")
    B, max_blocks = tshape
    num_slots = slot_mapping.nbytes >> 3
    keep = (block_table, lens_before, lens_after, free_blocks, placed, new_placed, cu_tokens, slot_mapping, positions)
    dev = block_table.get_device()
    # the common case in one expression (bytes cost a tensor less than its number of elements); the checks below only
    # name the failure
    if not (dev >= 0 and dev == _current_device()
            and _ready(dev, _I32, block_table, lens_before, lens_after, free_blocks, placed, new_placed, cu_tokens,
                       positions) and _ready(dev, _I64, slot_mapping)
            and lens_after.nbytes == 4 * B and cu_tokens.nbytes == 4 * B + 4 and placed.nbytes == 4
            and new_placed.nbytes == 4 and (lens_before is None or lens_before.nbytes == 4 * B)
            and (positions is None or positions.nbytes == 4 * num_slots)):
        num_slots = slot_mapping.numel()
        if lens_after.numel() != B or (lens_before is not None and lens_before.numel() != B) or cu_tokens.numel() != B + 1:
            raise ValueError("lens_before and lens_after must have B entries and cu_tokens B + 1")
        if placed.numel() != 1 or new_placed.numel() != 1:
            raise ValueError("placed and new_placed must have one entry")
        if positions is not None and positions.numel() != num_slots:
            raise ValueError("positions must have slot_mapping's size")
        _check_all(keep, (block_table, _I32, "block_table"), (lens_before, _I32, "lens_before"),
                   (lens_after, _I32, "lens_after"), (free_blocks, _I32, "free_blocks"), (placed, _I32, "placed"),
                   (new_placed, _I32, "new_placed"), (cu_tokens, _I32, "cu_tokens"),
                   (slot_mapping, _I64, "slot_mapping"), (positions, _I32, "positions"))
    args = (0 if lens_before is None else lens_before.data_ptr(), lens_after.data_ptr(), B, free_blocks.data_ptr(),
            free_blocks.nbytes >> 2, placed.data_ptr(), int(window), int(sinks), block_table.data_ptr(), max_blocks,
            int(block_size), new_placed.data_ptr(), cu_tokens.data_ptr(), slot_mapping.data_ptr(),
            0 if positions is None else positions.data_ptr(), num_slots)
    return _run(_BLOCK_TABLES, args, stream, prepare, dev, keep)


def _code_dtype(codes: torch.Tensor):
    """Codes come as torch.float8_e4m3fn or as their bytes."""
    if not isinstance(codes, torch.Tensor) or codes.dtype not in (_E4M3, _U8):
        raise TypeError("codes must be a torch.float8_e4m3fn or torch.uint8 tensor")
    return codes.dtype


def _code_shape(codes: torch.Tensor, scales: torch.Tensor, D: int):
    """(NB, Hkv, bs) of a block-scaled cache layer."""
    shape = codes.shape
    if len(shape) != 5:
        raise ValueError("codes must be [NB][Hkv][2][bs][D]")
    NB, Hkv, two, bs, Dk = shape
    if two != 2 or Dk != D or scales.shape != (NB, Hkv, 2):
        raise ValueError("codes must be [NB][Hkv][2][bs][D] and scales [NB][Hkv][2]")
    return NB, Hkv, bs


def kv_append_fp8_block(k_new: torch.Tensor, v_new: torch.Tensor, slot_mapping: torch.Tensor, codes: torch.Tensor,
                        scales: torch.Tensor, stream=None, prepare: bool = False):
    """Quantize k_new / v_new (fp16 [n][Hkv][D]; the tokens may be apart, as parts of one projection's output) into a
    block-scaled cache layer: codes [NB][Hkv][2][bs][D] (float8_e4m3fn or uint8: K's rows, V's rows) and scales float32
    [NB][Hkv][2], powers of two; slot_mapping int64 [n], the tokens of a block consecutive (see include/kvc.h).
    prepare=True returns a PreparedCall instead of launching."""
    kshape = k_new.shape
    if len(kshape) != 3 or v_new.shape != kshape:
        raise ValueError("k_new and v_new must be [n][Hkv][D]")
    n, Hkv, D = kshape
    NB, Hc, bs = _code_shape(codes, scales, D)
    if Hc != Hkv:
        raise ValueError("codes do not match k_new")
    dt = _code_dtype(codes)
    keep = (k_new, v_new, slot_mapping, codes, scales)
    dev = k_new.get_device()
    kst, vst = k_new.stride(), v_new.stride()
    if not (dev >= 0 and dev == _current_device() == v_new.get_device() and k_new.dtype is _F16 and v_new.dtype is _F16
            and kst[2] == vst[2] == 1 and kst[1] == vst[1] == D and _ready(dev, _I64, slot_mapping)
            and slot_mapping.nbytes == 8 * n and _ready(dev, dt, codes) and _ready(dev, _F32, scales)):
        if slot_mapping.numel() != n:
            raise ValueError("slot_mapping must have n entries")
        kst, vst = ((_token_stride(t, nm),) for t, nm in ((k_new, "k_new"), (v_new, "v_new")))
        _check_all(keep, (slot_mapping, _I64, "slot_mapping"), (codes, dt, "codes"), (scales, _F32, "scales"))
    if n == 1:  # a single token's stride means nothing
        kst, vst = (Hkv * D,), (Hkv * D,)
    args = (k_new.data_ptr(), kst[0], v_new.data_ptr(), vst[0], n, slot_mapping.data_ptr(), codes.data_ptr(),
            scales.data_ptr(), NB, Hkv, D, bs)
    return _run(_APPEND_FP8_BLOCK, args, stream, prepare, dev, keep)


def paged_decode_fp8_block_plan(B: int, Hq: int, Hkv: int, head_dim: int, max_context_len: int, window: int = 0,
                                sinks: int = 0, block_size: int = 16) -> int:
    """Workspace bytes of paged_decode_attention_fp8_block for these sizes."""
    ws = ctypes.c_size_t()
    _check(_lib.paged_decode_fp8_block_plan(B, Hq, Hkv, head_dim, block_size, max_context_len, int(window), int(sinks),
                                            ctypes.byref(ws)), "paged_decode_fp8_block_plan")
    return ws.value


def _check_decode_shapes(q, block_table, context_lens, out) -> None:
    """q, tables, lengths and out of a decode call agree."""
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    tshape = block_table.shape
    if len(tshape) != 2 or tshape[0] != q.shape[0] or context_lens.numel() != q.shape[0]:
        raise ValueError("block_table / context_lens do not match B")
    if out.dtype not in (_F16, _F32):
        raise TypeError("out must be float16 or float32")


def paged_decode_attention_fp8_block(q: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                                     block_table: torch.Tensor, context_lens: torch.Tensor, scale: float,
                                     out: torch.Tensor, workspace: Optional[torch.Tensor], max_context_len: int,
                                     window: int = 0, sinks: int = 0, stream=None, prepare: bool = False):
    """paged_decode_attention over a block-scaled cache layer (codes and scales as kv_append_fp8_block writes them), of
    all of a context (window 0) or of its newest `window` and first `sinks` positions; workspace:
    paged_decode_fp8_block_plan bytes.  prepare=True returns a PreparedCall instead of launching."""
    qshape, cshape, tshape = q.shape, codes.shape, block_table.shape
    B, Hq, D = qshape
    dt, odt = codes.dtype, out.dtype
    keep = (q, codes, scales, block_table, context_lens, out, workspace)
    dev = q.get_device()
    # the common case in one expression, written out (a call per tensor takes half as long again); the checks below only
    # name the failure
    if not (len(cshape) == 5 and len(tshape) == 2 and cshape[2] == 2 and cshape[4] == D and tshape[0] == B
            and scales.shape == (cshape[0], cshape[1], 2) and out.shape == qshape and context_lens.nbytes == 4 * B
            and dev >= 0 and dev == _current_device() and q.dtype is _F16 and (dt is _E4M3 or dt is _U8)
            and scales.dtype is _F32 and block_table.dtype is _I32 and context_lens.dtype is _I32
            and (odt is _F16 or odt is _F32)
            and dev == codes.get_device() == scales.get_device() == block_table.get_device()
            == context_lens.get_device() == out.get_device()
            and q.is_contiguous() and codes.is_contiguous() and scales.is_contiguous() and block_table.is_contiguous()
            and context_lens.is_contiguous() and out.is_contiguous()
            and (workspace is None or (workspace.get_device() == dev and workspace.is_contiguous()))):
        _code_shape(codes, scales, D)
        _check_decode_shapes(q, block_table, context_lens, out)
        dt = _code_dtype(codes)
        _check_all(keep, (q, _F16, "q"), (codes, dt, "codes"), (scales, _F32, "scales"),
                   (block_table, _I32, "block_table"), (context_lens, _I32, "context_lens"), (out, None, "out"),
                   (workspace, None, "workspace"))
    args = (q.data_ptr(), codes.data_ptr(), scales.data_ptr(), cshape[0], block_table.data_ptr(), tshape[1],
            context_lens.data_ptr(), int(window), int(sinks), B, Hq, cshape[1], D, cshape[3], int(max_context_len),
            float(scale), out.data_ptr(), KVC_F16 if odt is _F16 else KVC_F32, 0 if workspace is None else workspace.data_ptr(),
            0 if workspace is None else workspace.nbytes)
    return _run(_ATTENTION_FP8_BLOCK, args, stream, prepare, dev, keep)


def paged_decode_window_plan(B: int, Hq: int, Hkv: int, head_dim: int, max_context_len: int, window: int,
                             sinks: int = 0, block_size: int = 16) -> int:
    """Workspace bytes of paged_decode_window_attention for these sizes."""
    ws = ctypes.c_size_t()
    _check(_lib.paged_decode_window_plan(B, Hq, Hkv, head_dim, block_size, max_context_len, int(window), int(sinks),
                                         ctypes.byref(ws)), "paged_decode_window_plan")
    return ws.value


def paged_decode_window_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                  block_table: torch.Tensor, context_lens: torch.Tensor, window: int, sinks: int,
                                  scale: float, out: torch.Tensor, workspace: Optional[torch.Tensor],
                                  max_context_len: int, k_new: Optional[torch.Tensor] = None,
                                  v_new: Optional[torch.Tensor] = None, stream=None, prepare: bool = False):
    """paged_decode_attention over the newest `window` positions of every sequence and its first `sinks`; with
    k_new / v_new ([B][Hkv][D] fp16) these are appended at position ctx-1 first, in the same kernel.  Blocks in which
    nothing is visible are not read, nor their table entries; workspace: paged_decode_window_plan bytes.
    prepare=True returns a PreparedCall instead of launching."""
    qshape, cshape, tshape = q.shape, k_cache.shape, block_table.shape
    B, Hq, D = qshape
    NB, Hkv, bs, Dk = cshape
    if Dk != D or v_cache.shape != cshape:
        raise ValueError("cache shapes do not match q")
    odt = out.dtype
    if (k_new is None) != (v_new is None):
        raise ValueError("k_new and v_new: both or neither")
    if k_new is not None and (k_new.shape != (B, Hkv, D) or v_new.shape != (B, Hkv, D)):
        raise ValueError("k_new/v_new must be [B][Hkv][D]")
    keep = (q, k_cache, v_cache, block_table, context_lens, out, workspace, k_new, v_new)
    dev = q.get_device()
    # (as in paged_decode_attention_fp8_block)
    if not (len(tshape) == 2 and tshape[0] == B and out.shape == qshape and context_lens.nbytes == 4 * B
            and dev >= 0 and dev == _current_device() and q.dtype is k_cache.dtype is v_cache.dtype is _F16
            and block_table.dtype is _I32 and context_lens.dtype is _I32 and (odt is _F16 or odt is _F32)
            and dev == k_cache.get_device() == v_cache.get_device() == block_table.get_device()
            == context_lens.get_device() == out.get_device()
            and q.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous() and block_table.is_contiguous()
            and context_lens.is_contiguous() and out.is_contiguous()
            and (k_new is None or _ready(dev, _F16, k_new, v_new))
            and (workspace is None or (workspace.get_device() == dev and workspace.is_contiguous()))):
        _check_decode_shapes(q, block_table, context_lens, out)
        _check_all(keep, (q, _F16, "q"), (k_cache, _F16, "k_cache"), (v_cache, _F16, "v_cache"),
                   (k_new, _F16, "k_new"), (v_new, _F16, "v_new"), (block_table, _I32, "block_table"),
                   (context_lens, _I32, "context_lens"), (out, None, "out"), (workspace, None, "workspace"))
    args = (q.data_ptr(), 0 if k_new is None else k_new.data_ptr(), 0 if v_new is None else v_new.data_ptr(),
            k_cache.data_ptr(), v_cache.data_ptr(), NB, block_table.data_ptr(), tshape[1],
            context_lens.data_ptr(), int(window), int(sinks), B, Hq, Hkv, D, bs, int(max_context_len), float(scale),
            out.data_ptr(), KVC_F16 if odt is _F16 else KVC_F32, 0 if workspace is None else workspace.data_ptr(),
            0 if workspace is None else workspace.nbytes)
    return _run(_WINDOW_ATTENTION, args, stream, prepare, dev, keep)


def prefill_window_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                             max_seqlen: int, window: int, sinks: int, scale: float, out: torch.Tensor, stream=None,
                             precise: bool = False, prepare: bool = False):
    """Packed varlen prefill, causal, each row over the newest `window` rows of its segment and the first `sinks`:
    q [T][Hq][D], k/v [T][Hkv][D] fp16, cu_seqlens int32 [nseq+1] -> out [T][Hq][D] fp16 or fp32.  precise as in
    prefill_attention.  prepare=True returns a PreparedCall instead of launching."""
    qshape, kshape = q.shape, k.shape
    T, Hq, D = qshape
    if len(kshape) != 3 or kshape[0] != T or kshape[2] != D or v.shape != kshape or out.shape != qshape:
        raise ValueError("shape mismatch")
    Hkv = kshape[1]
    od = KVC_F16 if out.dtype is _F16 else KVC_F32 if out.dtype is _F32 else None
    if od is None:
        raise TypeError("out must be float16 or float32")
    keep = (q, k, v, cu_seqlens, out)
    dev = q.get_device()
    if not (dev >= 0 and dev == _current_device() and _ready(dev, _F16, q, k, v) and _ready(dev, _I32, cu_seqlens)
            and _ready(dev, out.dtype, out)):
        _check_all(keep, (q, _F16, "q"), (k, _F16, "k"), (v, _F16, "v"), (cu_seqlens, _I32, "cu_seqlens"),
                   (out, None, "out"))
    args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_seqlens.data_ptr(), cu_seqlens.numel() - 1, T, int(max_seqlen),
            Hq, Hkv, D, float(scale), int(window), int(sinks), KVC_PREFILL_P_SPLIT if precise else KVC_PREFILL_P_F16,
            out.data_ptr(), od)
    return _run(_PREFILL_WINDOW, args, stream, prepare, dev, keep)
