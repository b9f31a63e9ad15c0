"""Thin ctypes binding of the C ABI in include/hisparse_swap.h.

Every function here only marshals arguments (tensor pointers, sizes, the
current CUDA stream) and calls the library of the same name; all work runs
in the library's CUDA kernels.  There is no fallback: if the library has not
been built for this machine, loading it raises.

Tensors: device tensors are torch CUDA tensors, host pools are pinned torch
CPU tensors (``pin_memory=True``); all must be contiguous.
"""
from __future__ import annotations

import ctypes
import os
import re
import struct
import threading
from typing import Dict, List, Optional, Sequence

from . import build as _build

HS_OK = 0
HS_ERR_INVALID_ARG = -1
HS_ERR_UNSUPPORTED = -2
HS_ERR_CUDA = -3
HS_ERR_DEVICE_STATUS = -4
HS_ERR_TIMEOUT = -5

HS_STATUS_BAD_REQUEST = 0x1
HS_STATUS_DUPLICATE_REQUEST = 0x2
HS_STATUS_SEQ_LEN_CLAMPED = 0x4
HS_STATUS_PROBE_LIMIT = 0x8
HS_STATUS_TABLE_FULL = 0x10
HS_STATUS_BAD_APPEND = 0x20
HS_STATUS_BAD_PLAN = 0x40

HS_INDEX_HASH = 0
HS_INDEX_DENSE = 1

HS_STAT_EXTRA = 8
HS_NUM_STATS = 9
STAT_NAMES = ("hits", "hit_slots", "dup_misses", "unique_misses", "admitted", "evicted",
              "overflow", "invalid", "extra")
HS_MAX_EXTRA_PAGE = 65536
HS_MAX_ITEM_BYTES = 65536
HS_NOALLOC_SCRATCH_BYTES = 16 << 20
TIMELINE_WORDS_PER_ROW = 8 * 16  # hs_set_timeline: [batch][8 ranks][16 words]

HS_KV_E4M3 = 0
HS_KV_INT8 = 1
HS_DTYPE_BF16 = 0
HS_DTYPE_FP16 = 1
HS_DTYPE_FP32 = 2
HS_MAX_KV_BLOCK = 4096
HS_MAX_KV_HEADS = 128
HS_MAX_ROPE_AXES = 4
HS_MAX_SELECT_BLOCKS = 16384
HS_MAX_SELECT_WIDTH = 8192
HS_MAX_PREFIXES = 256

HEADER = os.path.join(_build.INCLUDE, "hisparse_swap.h")


class HsError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__("%s failed: %s (%d)" % (where, status_string(code), code))


class HsConfig(ctypes.Structure):
    _fields_ = [("num_requests", ctypes.c_int32), ("max_seq_len", ctypes.c_int32),
                ("item_size_bytes", ctypes.c_int32), ("hot_buffer_size", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("max_steps", ctypes.c_int32),
                ("num_layers", ctypes.c_int32), ("max_batch", ctypes.c_int32),
                ("index_kind", ctypes.c_int32), ("extra_page_size", ctypes.c_int32)]

    def as_dict(self) -> Dict[str, int]:
        return {name: getattr(self, name) for name, _ in self._fields_}


def make_config(num_requests: int, max_seq_len: int, item_size_bytes: int,
                hot_buffer_size: int, top_k: int, max_steps: int, num_layers: int = 1,
                max_batch: Optional[int] = None, index_kind: int = 0,
                extra_page_size: int = 0) -> HsConfig:
    """index_kind: HS_INDEX_HASH (0, hash banks) or HS_INDEX_DENSE (1, dense map);
    extra_page_size: rows of each request's extra page (0 = none)."""
    return HsConfig(num_requests, max_seq_len, item_size_bytes, hot_buffer_size, top_k,
                    max_steps, num_layers, num_requests if max_batch is None else max_batch,
                    index_kind, extra_page_size)


class HsKvFormat(ctypes.Structure):
    """Content of a KV row: 8-bit keys and values, a scale per block of tokens and head."""
    _fields_ = [("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("block_tokens", ctypes.c_int32), ("code", ctypes.c_int32),
                ("item_size_bytes", ctypes.c_int32)]

    def num_blocks(self, max_seq_len: int) -> int:
        """Scale blocks of a sequence of max_seq_len tokens."""
        return -(-max_seq_len // self.block_tokens)

    def scales_shape(self, num_requests: int, max_seq_len: int):
        return (num_requests, self.num_blocks(max_seq_len), 2, self.num_kv_heads)


def make_kv_format(num_kv_heads: int, head_dim: int, block_tokens: int, code: int = HS_KV_E4M3,
                   item_size_bytes: Optional[int] = None) -> HsKvFormat:
    """code: HS_KV_E4M3 or HS_KV_INT8; item_size_bytes: the row's width, by default just
    its keys and values.  Raises HsError if the library does not take the format."""
    width = 2 * num_kv_heads * head_dim if item_size_bytes is None else item_size_bytes
    fmt = HsKvFormat(num_kv_heads, head_dim, block_tokens, code, width)
    _check(load_library().hs_kv_format_check(ctypes.byref(fmt)), "hs_kv_format_check")
    return fmt


class _HsKvInput(ctypes.Structure):
    _fields_ = [("k_dev", ctypes.c_void_p), ("v_dev", ctypes.c_void_p),
                ("dtype", ctypes.c_int32), ("k_stride", ctypes.c_int64 * 3),
                ("v_stride", ctypes.c_int64 * 3)]  # hs_kv_input


class _HsAttendArgs(ctypes.Structure):
    _fields_ = [("q_dev", ctypes.c_void_p), ("out_dev", ctypes.c_void_p),
                ("dtype", ctypes.c_int32), ("batch", ctypes.c_int32), ("steps", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("num_requests", ctypes.c_int32), ("max_seq_len", ctypes.c_int32),
                ("sm_scale", ctypes.c_float), ("q_stride", ctypes.c_int64 * 3),
                ("out_stride", ctypes.c_int64 * 3), ("rows_dev", ctypes.c_void_p),
                ("num_rows", ctypes.c_int64), ("locs_dev", ctypes.c_void_p),
                ("topk_dev", ctypes.c_void_p), ("req_dev", ctypes.c_void_p),
                ("scales_dev", ctypes.c_void_p), ("lse_dev", ctypes.c_void_p),
                ("weights_dev", ctypes.c_void_p), ("acc_dev", ctypes.c_void_p),
                ("workspace_dev", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class _HsNormRopeArgs(ctypes.Structure):
    _fields_ = [("q_dev", ctypes.c_void_p), ("k_dev", ctypes.c_void_p),
                ("q_out_dev", ctypes.c_void_p), ("k_out_dev", ctypes.c_void_p),
                ("dtype", ctypes.c_int32), ("batch", ctypes.c_int32), ("tokens", ctypes.c_int32),
                ("num_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("adjacent", ctypes.c_int32), ("num_axes", ctypes.c_int32),
                ("eps", ctypes.c_float), ("q_stride", ctypes.c_int64 * 3),
                ("k_stride", ctypes.c_int64 * 3), ("q_out_stride", ctypes.c_int64 * 3),
                ("k_out_stride", ctypes.c_int64 * 3), ("q_weight_dev", ctypes.c_void_p),
                ("k_weight_dev", ctypes.c_void_p), ("pos_dev", ctypes.c_void_p),
                ("turns_dev", ctypes.c_void_p), ("axis_dev", ctypes.c_void_p),
                ("count_dev", ctypes.c_void_p)]


class _HsSelectArgs(ctypes.Structure):
    _fields_ = [("q_dev", ctypes.c_void_p), ("bounds_dev", ctypes.c_void_p),
                ("dtype", ctypes.c_int32), ("batch", ctypes.c_int32), ("steps", ctypes.c_int32),
                ("num_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("num_requests", ctypes.c_int32),
                ("max_seq_len", ctypes.c_int32), ("block_tokens", ctypes.c_int32),
                ("select", ctypes.c_int32), ("first", ctypes.c_int32), ("last", ctypes.c_int32),
                ("q_stride", ctypes.c_int64 * 3), ("req_dev", ctypes.c_void_p),
                ("seq_lens_dev", ctypes.c_void_p), ("blocks_dev", ctypes.c_void_p),
                ("topk_dev", ctypes.c_void_p), ("scores_dev", ctypes.c_void_p),
                ("workspace_dev", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class _HsPrefixArgs(ctypes.Structure):
    _fields_ = [("q_dev", ctypes.c_void_p), ("out_dev", ctypes.c_void_p),
                ("dtype", ctypes.c_int32), ("batch", ctypes.c_int32), ("steps", ctypes.c_int32),
                ("num_heads", ctypes.c_int32), ("num_requests", ctypes.c_int32),
                ("max_seq_len", ctypes.c_int32), ("num_prefixes", ctypes.c_int32),
                ("sm_scale", ctypes.c_float), ("q_stride", ctypes.c_int64 * 3),
                ("out_stride", ctypes.c_int64 * 3), ("join_stride", ctypes.c_int64 * 3),
                ("rows_dev", ctypes.c_void_p), ("scales_dev", ctypes.c_void_p),
                ("prefix_dev", ctypes.c_void_p), ("lens_dev", ctypes.c_void_p),
                ("starts_dev", ctypes.c_void_p), ("lse_dev", ctypes.c_void_p),
                ("join_out_dev", ctypes.c_void_p), ("join_lse_dev", ctypes.c_void_p),
                ("workspace_dev", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


_lib = None
_lock = threading.Lock()
_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_cfgp = ctypes.POINTER(HsConfig)
_fmtp = ctypes.POINTER(HsKvFormat)


def _declare(lib) -> None:
    sig = {
        "hs_config_check": (ctypes.c_int, [_cfgp]),
        "hs_state_bytes": (ctypes.c_size_t, [_cfgp]),
        "hs_workspace_bytes": (ctypes.c_size_t, [_cfgp]),
        "hs_device_kv_bytes": (ctypes.c_size_t, [_cfgp]),
        "hs_host_pool_bytes": (ctypes.c_size_t, [_cfgp]),
        "hs_hash_size": (_i32, [_cfgp]),
        "hs_create_state": (ctypes.c_int, [_cfgp, _vp, _vp, _vp, ctypes.c_size_t, _vp,
                                           ctypes.c_size_t, _vp, ctypes.POINTER(_vp)]),
        "hs_destroy_state": (None, [_vp]),
        "hs_swap_in": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp,
                                      _vp, _vp]),
        "hs_page_table": (ctypes.c_int, [_vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp,
                                         _vp]),
        "hs_reset_requests": (ctypes.c_int, [_vp, _vp, _i32, _vp]),
        "hs_get_status": (ctypes.c_int, [_vp, ctypes.POINTER(ctypes.c_uint32), _vp]),
        "hs_get_stats": (ctypes.c_int, [_vp, _i32, _vp, _i32, _vp]),
        "hs_export_request_state": (ctypes.c_int, [_vp, _i32, _i32, _vp, _vp, _vp, _vp, _vp,
                                                   _vp]),
        "hs_swap_in_noalloc": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp,
                                              _vp, _vp, _vp, _vp]),
        "hs_append_rows": (ctypes.c_int, [_vp, _i32, _vp, _vp, _vp, _vp, _i32, _vp]),
        "hs_set_timeline": (ctypes.c_int, [_vp, _vp]),
        "hs_set_defer_copy": (ctypes.c_int, [_vp, _i32]),
        "hs_copy_planned": (ctypes.c_int, [_vp, _i32, _vp, _vp, _vp, _i32, _vp]),
        "hs_set_copy_ctas": (ctypes.c_int, [_vp, _i32]),
        "hs_kv_format_check": (ctypes.c_int, [_fmtp]),
        "hs_quantize_kv": (ctypes.c_int, [_fmtp, _vp, _vp, _vp, _vp, _i32, _i32, _vp, _vp, _i32,
                                          _i32, _vp]),
        "hs_append_kv": (ctypes.c_int, [_vp, _i32, _fmtp, _vp, _vp, _vp, _vp, _i32, _i32, _vp,
                                        _vp]),
        "hs_attend_workspace_bytes": (ctypes.c_size_t, [_fmtp, _vp]),
        "hs_attend": (ctypes.c_int, [_fmtp, _vp, _vp]),
        "hs_accumulate": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _i32, _i32,
                                         _vp]),
        "hs_evict": (ctypes.c_int, [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp,
                                    _vp]),
        "hs_compact_kv": (ctypes.c_int, [_fmtp, _vp, _vp, _i32, _i32, _vp, _vp, _vp, _i32, _i32,
                                         _vp, _vp, _i32, _i32, _vp, _vp]),
        "hs_norm_rope": (ctypes.c_int, [_vp, _vp]),
        "hs_bound_keys": (ctypes.c_int, [_vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _i32,
                                         _i32, _vp, _i32, _i32, _vp]),
        "hs_select_workspace_bytes": (ctypes.c_size_t, [_i32, _i32, _i32, _i32]),
        "hs_select_blocks": (ctypes.c_int, [_vp, _vp]),
        "hs_prefix_workspace_bytes": (ctypes.c_size_t, [_fmtp, _vp]),
        "hs_attend_prefix": (ctypes.c_int, [_fmtp, _vp, _vp]),
        "hs_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "hs_version": (_i32, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args


def load_library(path: Optional[str] = None, build_if_missing: bool = False):
    """Load the in-tree library (optionally building it first)."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or _build.lib_path()
        if not os.path.exists(p):
            if not build_if_missing:
                raise RuntimeError("CUDA library %s is not built; run __graft_entry__.build() or "
                                   "python -m sparse_attention_kv_swap_gb300.build" % p)
            p = _build.build()
        lib = ctypes.CDLL(p)
        _declare(lib)
        if path is None:
            _lib = lib
        return lib


def header_symbols(header: str = HEADER) -> List[str]:
    """Names of the functions the public header declares."""
    with open(header) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(hs_[a-z_0-9]+)\s*\(", text)))


def status_string(code: int) -> str:
    try:
        return load_library().hs_status_string(code).decode()
    except Exception:
        return "status %d" % code


def _check(code: int, where: str) -> None:
    if code != HS_OK:
        raise HsError(code, where)


def _stream_ptr(stream) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    want = getattr(_call_device, "index", None)
    if want is not None and stream.device.index != want:
        raise ValueError("the stream is on cuda:%d, the call runs on cuda:%d"
                         % (stream.device.index, want))
    return int(stream.cuda_stream)


_call_device = threading.local()  # device of the handle whose call is being marshalled


class _on_device:
    """Makes device `index` current for one library call (a handle's calls
    must be made on its own device) and has _dptr and _stream_ptr reject
    device tensors and streams of another device.  `index` None checks and
    switches nothing."""

    def __init__(self, index: Optional[int]):
        self.index = index

    def __enter__(self):
        import torch
        self.outer = getattr(_call_device, "index", None)
        _call_device.index = self.index
        self.prev = None
        if self.index is not None and torch.cuda.is_available():
            prev = torch.cuda.current_device()
            if prev != self.index:
                torch.cuda.set_device(self.index)
                self.prev = prev
        return self

    def __exit__(self, *exc):
        _call_device.index = self.outer
        if self.prev is not None:
            torch.cuda.set_device(self.prev)
        return False


def _dptr(t, dtype=None, name="tensor") -> int:
    """Address of a tensor the kernels read or write: device memory, or pinned
    (mapped) host memory, which the device addresses directly.  Inside
    _on_device, a device tensor must be on that device."""
    if t is None:
        return 0
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must have dtype %s" % (name, dtype))
    if not (t.is_cuda or t.is_pinned()):
        raise ValueError("%s must be in device memory or pinned host memory" % name)
    want = getattr(_call_device, "index", None)
    if t.is_cuda and want is not None and t.device.index != want:
        raise ValueError("%s is on cuda:%d, the call runs on cuda:%d" % (name, t.device.index,
                                                                        want))
    return int(t.data_ptr())


def _hptr(t, name="tensor") -> int:
    """Address of a host pool: pinned, or pageable where the library accepts it
    (it checks the memory kind itself)."""
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return int(t.data_ptr())


def _shape(t, shape, name) -> None:
    """The kernels trust the sizes: check them before any launch."""
    if t is not None and t.shape != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def _swap_in_shapes(handle, req_pool_indices, seq_lens, topk, device_locs, stats, miss_src,
                    miss_dst, miss_count):
    if topk.dim() != 3:
        raise ValueError("topk must be [batch, steps, top_k]")
    B, S, K = topk.shape
    cfg = handle.cfg
    if K != cfg.top_k:
        raise ValueError("topk's last dimension %d differs from the config's top_k %d"
                         % (K, cfg.top_k))
    C = cfg.max_steps * cfg.top_k
    _shape(req_pool_indices, (B,), "req_pool_indices")
    _shape(seq_lens, (B,), "seq_lens")
    _shape(device_locs, (B, S, K), "device_locs")
    _shape(stats, (B, HS_NUM_STATS), "stats")
    _shape(miss_src, (B, C), "miss_src")
    _shape(miss_dst, (B, C), "miss_dst")
    _shape(miss_count, (B,), "miss_count")
    return B, S, K


# ---- sizes -----------------------------------------------------------------

def hs_config_check(cfg: HsConfig) -> int:
    return load_library().hs_config_check(ctypes.byref(cfg))


def hs_state_bytes(cfg: HsConfig) -> int:
    return load_library().hs_state_bytes(ctypes.byref(cfg))


def hs_workspace_bytes(cfg: HsConfig) -> int:
    return load_library().hs_workspace_bytes(ctypes.byref(cfg))


def hs_device_kv_bytes(cfg: HsConfig) -> int:
    return load_library().hs_device_kv_bytes(ctypes.byref(cfg))


def hs_host_pool_bytes(cfg: HsConfig) -> int:
    return load_library().hs_host_pool_bytes(ctypes.byref(cfg))


def hs_hash_size(cfg: HsConfig) -> int:
    return load_library().hs_hash_size(ctypes.byref(cfg))


def hs_version() -> int:
    return load_library().hs_version()


def hs_status_string(code: int) -> str:
    return load_library().hs_status_string(code).decode()


# ---- state -------------------------------------------------------------------

class StateHandle:
    """Owns the library's host handle; keeps the caller's tensors alive."""

    def __init__(self, ptr: int, cfg: HsConfig, keep: Sequence, device: int):
        self.ptr = ctypes.c_void_p(ptr)
        self.cfg = cfg
        self.device = device  # the CUDA device the handle and its buffers are on
        self._keep = list(keep)

    def pool_ptr(self, t) -> Optional[int]:
        """Address of `t` if it is one of the handle's host pools (which may be pageable), or None."""
        at = t.data_ptr()
        return at if any(at == x.data_ptr() for x in self._keep[:self.cfg.num_layers]) else None

    def close(self) -> None:
        if self.ptr:
            load_library().hs_destroy_state(self.ptr)
            self.ptr = ctypes.c_void_p(0)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def hs_create_state(cfg: HsConfig, host_pools: Sequence, device_kvs: Sequence, state, workspace,
                    stream=None) -> StateHandle:
    lib = load_library()
    L = cfg.num_layers
    if len(host_pools) != L or len(device_kvs) != L:
        raise ValueError("need one host pool and one device KV buffer per layer")
    # The handle belongs to the device that holds its device buffers.
    if not state.is_cuda:
        raise ValueError("state must be in device memory")
    device = state.device.index
    with _on_device(device):
        hp = (ctypes.c_void_p * L)(*[_hptr(t, name="host pool") for t in host_pools])
        dk = (ctypes.c_void_p * L)(*[_dptr(t, name="device kv") for t in device_kvs])
        out = ctypes.c_void_p()
        rc = lib.hs_create_state(ctypes.byref(cfg), ctypes.cast(hp, _vp), ctypes.cast(dk, _vp),
                                 _dptr(state, name="state"), state.numel() * state.element_size(),
                                 _dptr(workspace, name="workspace"),
                                 workspace.numel() * workspace.element_size(),
                                 _stream_ptr(stream), ctypes.byref(out))
    _check(rc, "hs_create_state")
    return StateHandle(out.value, cfg, list(host_pools) + list(device_kvs) + [state, workspace],
                       device)


def hs_destroy_state(handle: StateHandle) -> None:
    handle.close()


def hs_swap_in(handle: StateHandle, req_pool_indices, seq_lens, topk, layer_id: int,
               device_locs, stats=None, miss_src=None, miss_dst=None, miss_count=None,
               stream=None) -> None:
    import torch
    B, S, K = _swap_in_shapes(handle, req_pool_indices, seq_lens, topk, device_locs, stats,
                              miss_src, miss_dst, miss_count)
    with _on_device(handle.device):
        rc = load_library().hs_swap_in(
            handle.ptr, _dptr(req_pool_indices, torch.int32, "req_pool_indices"),
            _dptr(seq_lens, torch.int32, "seq_lens"), _dptr(topk, torch.int32, "topk"), B, S,
            layer_id, _dptr(device_locs, torch.int32, "device_locs"),
            _dptr(stats, torch.int32, "stats"), _dptr(miss_src, torch.int64, "miss_src"),
            _dptr(miss_dst, torch.int64, "miss_dst"),
            _dptr(miss_count, torch.int32, "miss_count"), _stream_ptr(stream))
        _check(rc, "hs_swap_in")


def hs_page_table(topk, seq_lens, max_seq_len: int, page_size: int, pages, num_pages,
                  token_page, stream=None) -> None:
    import torch
    if topk.dim() != 3:
        raise ValueError("topk must be [batch, steps, top_k]")
    B, S, K = topk.shape
    _shape(seq_lens, (B,), "seq_lens")
    _shape(pages, (B, S * K), "pages")
    _shape(num_pages, (B,), "num_pages")
    _shape(token_page, (B, S, K), "token_page")
    # runs on the device of its inputs (the current device for pinned host inputs)
    with _on_device(topk.device.index if topk.is_cuda else None):
        rc = load_library().hs_page_table(
            _dptr(topk, torch.int32, "topk"), _dptr(seq_lens, torch.int32, "seq_lens"), B, S, K,
            max_seq_len, page_size, _dptr(pages, torch.int32, "pages"),
            _dptr(num_pages, torch.int32, "num_pages"), _dptr(token_page, torch.int32, "token_page"),
            _stream_ptr(stream))
        _check(rc, "hs_page_table")


def hs_reset_requests(handle: StateHandle, req_pool_indices, stream=None) -> None:
    import torch
    if req_pool_indices.dim() != 1:
        raise ValueError("req_pool_indices must be 1-D")
    with _on_device(handle.device):
        rc = load_library().hs_reset_requests(
            handle.ptr, _dptr(req_pool_indices, torch.int32, "req_pool_indices"),
            req_pool_indices.numel(), _stream_ptr(stream))
        _check(rc, "hs_reset_requests")


def hs_get_status(handle: StateHandle, stream=None):
    """Returns (code, flags); synchronises the stream and clears the flags."""
    flags = ctypes.c_uint32(0)
    with _on_device(handle.device):
        rc = load_library().hs_get_status(handle.ptr, ctypes.byref(flags), _stream_ptr(stream))
        if rc not in (HS_OK, HS_ERR_DEVICE_STATUS):
            _check(rc, "hs_get_status")
    return rc, flags.value


def hs_export_request_state(handle: StateHandle, layer_id: int, request: int, stream=None):
    import numpy as np
    cfg = handle.cfg
    H = cfg.hot_buffer_size
    C = cfg.max_steps * cfg.top_k
    tok = np.empty(H, np.int32)
    ep = np.empty(H, np.int32)
    phys = np.empty(H + C, np.int32)
    ctrl = np.empty(8, np.int32)
    # hash entries, or the dense map widened to int64 [max_seq_len]
    bank = np.empty(cfg.max_seq_len if cfg.index_kind == HS_INDEX_DENSE else hs_hash_size(cfg),
                    np.int64)
    with _on_device(handle.device):
        rc = load_library().hs_export_request_state(
            handle.ptr, layer_id, request, tok.ctypes.data, ep.ctypes.data, phys.ctypes.data,
            ctrl.ctypes.data, bank.ctypes.data, _stream_ptr(stream))
        _check(rc, "hs_export_request_state")
    return {"tok": tok, "ep": ep, "phys": phys, "ctrl": ctrl, "bank": bank,
            "epoch": int(ctrl[0])}


def hs_append_rows(handle: StateHandle, layer_id: int, req, tok, seq_lens, rows,
                   stream=None) -> None:
    """Write-back of newly decoded rows: req/tok/seq_lens int32 [n], rows uint8
    [n, W] on the device (see the C header)."""
    import torch
    n = req.numel()
    _shape(req, (n,), "req")
    _shape(tok, (n,), "tok")
    _shape(seq_lens, (n,), "seq_lens")
    _shape(rows, (n, handle.cfg.item_size_bytes), "rows")
    with _on_device(handle.device):
        rc = load_library().hs_append_rows(
            handle.ptr, layer_id, _dptr(req, torch.int32, "req"), _dptr(tok, torch.int32, "tok"),
            _dptr(seq_lens, torch.int32, "seq_lens"), _dptr(rows, torch.uint8, "rows"), n,
            _stream_ptr(stream))
        _check(rc, "hs_append_rows")


def hs_get_stats(handle: StateHandle, layer_id: int, reset: bool = False, stream=None):
    """Running sums of the HS_STAT_* counters of one layer: int64 [HS_NUM_STATS]."""
    import numpy as np
    out = np.zeros(HS_NUM_STATS, dtype=np.int64)
    with _on_device(handle.device):
        rc = load_library().hs_get_stats(handle.ptr, layer_id, out.ctypes.data, 1 if reset else 0,
                                         _stream_ptr(stream))
        _check(rc, "hs_get_stats")
    return out


def hs_set_timeline(handle: StateHandle, timeline=None) -> None:
    """timeline: a uint64-sized CUDA tensor of at least max_batch * 128
    elements on the handle's device (the per-CTA phase stamps of later
    swap-ins, [batch][8][16]), or None to stop recording."""
    import torch
    ptr = 0
    with _on_device(handle.device):
        if timeline is not None:
            if not timeline.is_cuda:
                raise ValueError("timeline must be in device memory")
            if timeline.numel() < handle.cfg.max_batch * TIMELINE_WORDS_PER_ROW:
                raise ValueError("timeline: need %d elements, got %d"
                                 % (handle.cfg.max_batch * TIMELINE_WORDS_PER_ROW,
                                    timeline.numel()))
            ptr = _dptr(timeline, torch.int64, "timeline")
        _check(load_library().hs_set_timeline(handle.ptr, ptr), "hs_set_timeline")


def hs_set_copy_ctas(handle: StateHandle, copy_ctas: int) -> None:
    _check(load_library().hs_set_copy_ctas(handle.ptr, copy_ctas), "hs_set_copy_ctas")


def hs_set_defer_copy(handle: StateHandle, defer: bool) -> None:
    _check(load_library().hs_set_defer_copy(handle.ptr, 1 if defer else 0), "hs_set_defer_copy")


def hs_copy_planned(handle: StateHandle, layer_id: int, miss_src, miss_dst, miss_count,
                    stream=None) -> None:
    import torch
    B = miss_count.numel()
    C = handle.cfg.max_steps * handle.cfg.top_k
    _shape(miss_count, (B,), "miss_count")
    _shape(miss_src, (B, C), "miss_src")
    _shape(miss_dst, (B, C), "miss_dst")
    with _on_device(handle.device):
        rc = load_library().hs_copy_planned(
            handle.ptr, layer_id, _dptr(miss_src, torch.int64, "miss_src"),
            _dptr(miss_dst, torch.int64, "miss_dst"), _dptr(miss_count, torch.int32, "miss_count"),
            miss_count.numel(), _stream_ptr(stream))
        _check(rc, "hs_copy_planned")


def hs_swap_in_noalloc(handle: StateHandle, req_pool_indices, seq_lens, topk, layer_id: int,
                       device_locs, stats=None, miss_src=None, miss_dst=None, miss_count=None,
                       stream=None) -> None:
    """hs_swap_in whose per-call scratch is the library's fixed device array
    (for callers that cannot allocate device memory); see the C header."""
    import torch
    B, S, K = _swap_in_shapes(handle, req_pool_indices, seq_lens, topk, device_locs, stats,
                              miss_src, miss_dst, miss_count)
    with _on_device(handle.device):
        rc = load_library().hs_swap_in_noalloc(
            handle.ptr, _dptr(req_pool_indices, torch.int32, "req_pool_indices"),
            _dptr(seq_lens, torch.int32, "seq_lens"), _dptr(topk, torch.int32, "topk"), B, S,
            layer_id, _dptr(device_locs, torch.int32, "device_locs"),
            _dptr(stats, torch.int32, "stats"), _dptr(miss_src, torch.int64, "miss_src"),
            _dptr(miss_dst, torch.int64, "miss_dst"),
            _dptr(miss_count, torch.int32, "miss_count"), _stream_ptr(stream))
        _check(rc, "hs_swap_in_noalloc")


# ---- 8-bit key/value rows ------------------------------------------------------
#
# These calls run once per layer and decode step, some for a few microseconds of GPU time:
# the checks below take the short way for what is right and leave the wording of errors to
# the helpers above.

_ATTEND_ARGS = struct.Struct("@PP7if3q3qPq8PN")  # hs_attend_args
_KV_INPUT = struct.Struct("@PPi3q3q")  # hs_kv_input


def _ptr(t, dtype, name, device) -> int:
    """_dptr for a call on `device`; None is a null pointer."""
    if t is None:
        return 0
    if t.dtype is dtype and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    outer = getattr(_call_device, "index", None)
    _call_device.index = device
    try:
        return _dptr(t, dtype, name)
    finally:
        _call_device.index = outer


def _sptr(t, name, device) -> int:
    """Address of a device tensor that the kernels read by strides; its last
    dimension must be dense."""
    d = t.get_device()
    if d < 0:
        raise ValueError("%s must be in device memory" % name)
    if d != device:
        raise ValueError("%s is on cuda:%d, the call runs on cuda:%d" % (name, d, device))
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError("the last dimension of %s must be dense" % name)
    return t.data_ptr()


def _device_of(t, name) -> int:
    d = t.get_device()
    if d < 0:
        raise ValueError("%s must be in device memory" % name)
    return d


def _raw_stream(stream, device) -> int:
    import torch
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    if stream.device.index != device:
        raise ValueError("the stream is on cuda:%d, the call runs on cuda:%d"
                         % (stream.device.index, device))
    return stream.cuda_stream


def _run(name, device, *args) -> None:
    """Calls the library with `device` current and raises on an error code."""
    import torch
    fn = getattr(_lib or load_library(), name)
    if torch._C._cuda_getDevice() == device:
        rc = fn(*args)
    else:
        with torch.cuda.device(device):
            rc = fn(*args)
    if rc != HS_OK:
        raise HsError(rc, name)


def _dtype_code(t, name, allow_fp32: bool) -> int:
    import torch
    d = t.dtype
    if d is torch.bfloat16:
        return HS_DTYPE_BF16
    if d is torch.float16:
        return HS_DTYPE_FP16
    if d is torch.float32 and allow_fp32:
        return HS_DTYPE_FP32
    raise ValueError("%s must have dtype bfloat16%s float16%s"
                     % ((name,) + ((",", " or float32") if allow_fp32 else (" or", ""))))


def _kv_input(fmt, k, v, req, start, count, device):
    """The packed hs_kv_input, batch and tokens."""
    shape = k.shape
    if len(shape) != 4 or shape[2] != fmt.num_kv_heads or shape[3] != fmt.head_dim:
        raise ValueError("k must be [batch, tokens, %d, %d], got %s"
                         % (fmt.num_kv_heads, fmt.head_dim, tuple(shape)))
    if v.shape != shape:
        _shape(v, shape, "v")
    if v.dtype is not k.dtype:
        raise ValueError("k and v must have one dtype")
    B = shape[:1]
    if req.shape != B or start.shape != B or count.shape != B:
        _shape(req, B, "req")
        _shape(start, B, "start")
        _shape(count, B, "count")
    ka, kb, kc, _ = k.stride()
    va, vb, vc, _ = v.stride()
    return _KV_INPUT.pack(_sptr(k, "k", device), _sptr(v, "v", device), _dtype_code(k, "k", True),
                          ka, kb, kc, va, vb, vc), B[0], shape[1]


def _store(fmt, rows, scales, name):
    """(requests, tokens) of a store of rows [requests, tokens, W] and its scales."""
    shape = rows.shape
    if len(shape) != 3 or shape[2] != fmt.item_size_bytes:
        raise ValueError("%srows must be [requests, tokens, %d], got %s"
                         % (name, fmt.item_size_bytes, tuple(shape)))
    R, L, _ = shape
    if scales.shape != (R, -(-L // fmt.block_tokens), 2, fmt.num_kv_heads):
        _shape(scales, fmt.scales_shape(R, L), name + "scales")
    return R, L


def hs_quantize_kv(fmt: HsKvFormat, k, v, req, start, count, rows, scales, stream=None) -> None:
    """Quantises tokens [start[b], start[b] + count[b]) of request req[b] into a
    store of rows.  k, v: [batch, tokens, Hkv, D] (bf16, fp16 or fp32, any strides
    but a dense last dimension); rows uint8 [R, L, W] (device or pinned memory);
    scales fp32 [R, NB, 2, Hkv], updated."""
    import torch
    R, L = _store(fmt, rows, scales, "")
    i32, dev = torch.int32, k.get_device()
    inp, B, M = _kv_input(fmt, k, v, req, start, count, dev)
    _run("hs_quantize_kv", dev, fmt, inp, _ptr(req, i32, "req", dev),
         _ptr(start, i32, "start", dev), _ptr(count, i32, "count", dev), B, M,
         _ptr(rows, torch.uint8, "rows", dev), _ptr(scales, torch.float32, "scales", dev), R, L,
         _raw_stream(stream, dev))


def hs_append_kv(handle: StateHandle, layer_id: int, fmt: HsKvFormat, k, v, req, start, count,
                 scales, stream=None) -> None:
    """hs_quantize_kv into every copy that a swap-in handle keeps of the rows (host
    pool, extra page, hot rows); scales fp32 [R, NB, 2, Hkv] of the layer, updated."""
    import torch
    cfg = handle.cfg
    _shape(scales, fmt.scales_shape(cfg.num_requests, cfg.max_seq_len), "scales")
    i32, dev = torch.int32, handle.device
    inp, B, M = _kv_input(fmt, k, v, req, start, count, dev)
    _run("hs_append_kv", dev, handle.ptr, layer_id, fmt, inp, _ptr(req, i32, "req", dev),
         _ptr(start, i32, "start", dev), _ptr(count, i32, "count", dev), B, M,
         _ptr(scales, torch.float32, "scales", dev), _raw_stream(stream, dev))


def hs_attend_workspace_bytes(fmt: HsKvFormat, batch: int, steps: int, top_k: int,
                              num_heads: int) -> int:
    """Device bytes of workspace that hs_attend needs for these sizes (mostly 0)."""
    args = _HsAttendArgs(batch=batch, steps=steps, top_k=top_k, num_heads=num_heads)
    n = load_library().hs_attend_workspace_bytes(fmt, ctypes.byref(args))
    if n == ctypes.c_size_t(-1).value:
        raise HsError(HS_ERR_INVALID_ARG, "hs_attend_workspace_bytes")
    return n


def hs_attend(fmt: HsKvFormat, q, rows, locs, topk, req, scales, max_seq_len: int, out, lse=None,
              weights=None, acc=None, sm_scale: Optional[float] = None, workspace=None,
              stream=None) -> None:
    """Attention of q [batch, steps, heads, D] (bf16 or fp16) over the rows at
    locs [batch, steps, top_k] of rows uint8 [..., W].  topk: the rows' positions, req
    [batch]: their requests, which select the scales [R, NB, 2, Hkv].  Outputs: out
    as q, lse fp32 [batch, steps, heads], weights fp32 [batch, steps, top_k], acc fp32
    [R, max_seq_len] added to.  sm_scale: 1 / sqrt(D) by default."""
    import torch
    W, shape, sel = fmt.item_size_bytes, q.shape, topk.shape
    if len(shape) != 4 or shape[3] != fmt.head_dim:
        raise ValueError("q must be [batch, steps, heads, %d], got %s"
                         % (fmt.head_dim, tuple(shape)))
    B, S, H, D = shape
    if len(sel) != 3 or sel[0] != B or sel[1] != S:
        raise ValueError("topk must be [%d, %d, top_k], got %s" % (B, S, tuple(sel)))
    if out.dtype is not q.dtype:
        raise ValueError("out must have q's dtype")
    R = scales.shape[0] if scales.dim() else 0
    if (out.shape != shape or locs.shape != sel or req.shape != shape[:1]
            or scales.shape != (R, -(-max_seq_len // fmt.block_tokens), 2, fmt.num_kv_heads)):
        _shape(out, shape, "out")
        _shape(locs, sel, "locs")
        _shape(req, (B,), "req")
        if scales.dim() != 4:
            raise ValueError("scales must be [requests, blocks, 2, heads]")
        _shape(scales, fmt.scales_shape(R, max_seq_len), "scales")
    if lse is not None and lse.shape != shape[:3]:
        _shape(lse, (B, S, H), "lse")
    if weights is not None and weights.shape != sel:
        _shape(weights, sel, "weights")
    if acc is not None and acc.shape != (R, max_seq_len):
        _shape(acc, (R, max_seq_len), "acc")
    if rows.shape[-1] != W:
        raise ValueError("rows must be %d bytes wide" % W)
    i32, f32, dev = torch.int32, torch.float32, q.get_device()
    qa, qb, qc, _ = q.stride()
    oa, ob, oc, _ = out.stride()
    args = _ATTEND_ARGS.pack(
        _sptr(q, "q", dev), _sptr(out, "out", dev), _dtype_code(q, "q", False), B, S, sel[2], H, R,
        max_seq_len, D ** -0.5 if sm_scale is None else sm_scale, qa, qb, qc, oa, ob, oc,
        _ptr(rows, torch.uint8, "rows", dev), rows.numel() // W,
        _ptr(locs, i32, "locs", dev), _ptr(topk, i32, "topk", dev), _ptr(req, i32, "req", dev),
        _ptr(scales, f32, "scales", dev), _ptr(lse, f32, "lse", dev),
        _ptr(weights, f32, "weights", dev), _ptr(acc, f32, "acc", dev),
        0 if workspace is None else _ptr(workspace, workspace.dtype, "workspace", dev),
        0 if workspace is None else workspace.numel() * workspace.element_size())
    _run("hs_attend", dev, fmt, args, _raw_stream(stream, dev))


def hs_accumulate(weights, topk, req, acc, counts=None, stream=None) -> None:
    """acc[req[b], topk[b, s, j]] += weights[b, s, j] for the first counts[b] steps
    (all by default).  weights fp32 and topk int32 [batch, steps, top_k], acc fp32 [R, L]."""
    import torch
    if topk.dim() != 3:
        raise ValueError("topk must be [batch, steps, top_k]")
    B, S, K = topk.shape
    _shape(weights, (B, S, K), "weights")
    _shape(req, (B,), "req")
    _shape(counts, (B,), "counts")
    if acc.dim() != 2:
        raise ValueError("acc must be [requests, tokens]")
    i32, f32, dev = torch.int32, torch.float32, _device_of(acc, "acc")
    _run("hs_accumulate", dev,
         _ptr(weights, f32, "weights", dev), _ptr(topk, i32, "topk", dev),
         _ptr(req, i32, "req", dev), _ptr(counts, i32, "counts", dev), B, S, K,
         _ptr(acc, f32, "acc", dev), acc.shape[0], acc.shape[1], _raw_stream(stream, dev))


def hs_evict(acc, req, seq_lens, recent: int, keep, kept, kept_acc=None, stream=None) -> None:
    """Chooses the tokens that each request keeps: keep int32 [batch, budget] and kept
    int32 [batch] (out), kept_acc fp32 [batch, budget] (out) from acc fp32 [R, L]."""
    import torch
    if acc.dim() != 2 or keep.dim() != 2:
        raise ValueError("acc must be [requests, tokens] and keep [batch, budget]")
    shape = keep.shape
    (B, budget), one = shape, shape[:1]
    if req.shape != one or seq_lens.shape != one or kept.shape != one:
        _shape(req, one, "req")
        _shape(seq_lens, one, "seq_lens")
        _shape(kept, one, "kept")
    if kept_acc is not None and kept_acc.shape != shape:
        _shape(kept_acc, shape, "kept_acc")
    R, L = acc.shape
    i32, f32, dev = torch.int32, torch.float32, _device_of(acc, "acc")
    _run("hs_evict", dev, _ptr(acc, f32, "acc", dev),
         _ptr(req, i32, "req", dev), _ptr(seq_lens, i32, "seq_lens", dev), B, recent, budget,
         R, L, _ptr(keep, i32, "keep", dev), _ptr(kept, i32, "kept", dev),
         _ptr(kept_acc, f32, "kept_acc", dev), _raw_stream(stream, dev))


def hs_compact_kv(fmt: HsKvFormat, src_rows, src_scales, src_req, keep, kept, dst_rows,
                  dst_scales, dst_req, stream=None, handle: Optional[StateHandle] = None) -> None:
    """Moves the kept tokens (hs_evict's keep and kept) of requests src_req of one
    store of rows to the first places of requests dst_req of another.  src_rows that are a
    host pool of `handle` may be of any memory that the handle has accepted."""
    import torch
    sR, sL = _store(fmt, src_rows, src_scales, "src_")
    dR, dL = _store(fmt, dst_rows, dst_scales, "dst_")
    if keep.dim() != 2:
        raise ValueError("keep must be [batch, budget]")
    shape = keep.shape
    (B, budget), one = shape, shape[:1]
    if kept.shape != one or src_req.shape != one or dst_req.shape != one:
        _shape(kept, one, "kept")
        _shape(src_req, one, "src_req")
        _shape(dst_req, one, "dst_req")
    i32, f32, u8, dev = torch.int32, torch.float32, torch.uint8, _device_of(keep, "keep")
    src = handle.pool_ptr(src_rows) if handle is not None else None
    if src is None:
        src = _ptr(src_rows, u8, "src_rows", dev)
    _run("hs_compact_kv", dev, fmt, src, _ptr(src_scales, f32, "src_scales", dev), sR, sL,
         _ptr(src_req, i32, "src_req", dev), _ptr(keep, i32, "keep", dev),
         _ptr(kept, i32, "kept", dev), B, budget, _ptr(dst_rows, u8, "dst_rows", dev),
         _ptr(dst_scales, f32, "dst_scales", dev), dR, dL, _ptr(dst_req, i32, "dst_req", dev),
         _raw_stream(stream, dev))


# ---- around a decode step: norms and rotation, block selection, shared prefix ----

_NORM_ROPE_ARGS = struct.Struct("@4P9if3q3q3q3q6P")  # hs_norm_rope_args
_STRIDES = struct.Struct("@3q")
_SELECT_ARGS = struct.Struct("@PP12i3q6PN")  # hs_select_args
_PREFIX_ARGS = struct.Struct("@PP7if3q3q3q9PN")  # hs_prefix_args
_NO_SIZES = ctypes.c_size_t(-1).value


class HsRope:
    """Frequencies of a position rotation on one device (make_rope)."""

    def __init__(self, turns, axis, rot_dim: int, num_axes: int, adjacent: bool):
        self.turns, self.axis = turns, axis  # int64 and int32 [rot_dim / 2]; axis None: all 0
        self.rot_dim, self.num_axes, self.adjacent = rot_dim, num_axes, adjacent


def make_rope(inv_freq, axis=None, adjacent: bool = False, device=None) -> HsRope:
    """inv_freq: radians per position of each pair (floats or a 64-bit tensor), a multiple of 8
    of them; axis: the position axis of each pair (all 0 by default); adjacent: pairs are
    (2 j, 2 j + 1) instead of (j, j + rot_dim / 2)."""
    import math
    import torch
    freq = [float(f) for f in inv_freq]
    axis = None if axis is None else [int(x) for x in axis]
    if len(freq) % 8 or not all(math.isfinite(f) for f in freq):
        raise ValueError("inv_freq must be a multiple of 8 finite numbers")
    if axis is not None and (len(axis) != len(freq)
                             or any(not 0 <= x < HS_MAX_ROPE_AXES for x in axis)):
        raise ValueError("axis must give an axis from 0 to %d for every pair"
                         % (HS_MAX_ROPE_AXES - 1))
    # parts of a turn in 64-bit fixed point, whole turns dropped
    turns = [round(math.fmod(f / (2 * math.pi), 1.0) * 2.0 ** 64) % 2 ** 64 for f in freq]
    turns = [x - 2 ** 64 if x >= 2 ** 63 else x for x in turns]
    device = torch.device(device or "cuda")
    num_axes = 1 + max(axis, default=0) if axis else 1
    if num_axes == 1:
        axis = None
    return HsRope(torch.tensor(turns, dtype=torch.int64, device=device),
                  None if axis is None else torch.tensor(axis, dtype=torch.int32, device=device),
                  2 * len(freq), num_axes, bool(adjacent))


def _heads(t, name, batch_tokens=None, dim=None):
    """Shape of a tensor [batch, tokens, heads, D] (dense last dimension)."""
    shape = t.shape
    if len(shape) != 4 or (dim is not None and shape[3] != dim) or (
            batch_tokens is not None and shape[:2] != batch_tokens):
        raise ValueError("%s must be [batch, tokens, heads, head_dim]%s, got %s"
                         % (name, "" if dim is None else " with %s and head_dim %d"
                            % (tuple(batch_tokens), dim), tuple(shape)))
    return shape


def hs_norm_rope(q, k, positions, rope: Optional[HsRope], q_out, k_out, q_weight=None,
                 k_weight=None, eps: float = 1e-6, count=None, stream=None) -> None:
    """Norms of the heads of q [batch, tokens, heads, D] and k [batch, tokens, kv heads, D] (bf16,
    fp16 or fp32; either may be None), each if its weight (fp32 [D]) is given, and the rotation
    by positions int32 [axes, batch, tokens] ([batch, tokens] for one axis; rope None: no
    rotation) into q_out and k_out, which may be q and k.  count int32 [batch]: tokens
    of each entry."""
    import torch
    one = q if q is not None else k
    if one is None:
        raise ValueError("q or k must be given")
    B, M, _, D = _heads(one, "q" if q is not None else "k")
    dev, i32, f32 = one.get_device(), torch.int32, torch.float32
    sides, ptrs, strides, heads = ((q, q_out, "q"), (k, k_out, "k")), [], [], []
    for t, out, name in sides:
        if (t is None) != (out is None):
            raise ValueError("%s and %s_out must be given together" % (name, name))
        if t is None:
            ptrs.append((0, 0))
            strides.append(((0, 0, 0), (0, 0, 0)))
            heads.append(0)
            continue
        shape = _heads(t, name, one.shape[:2], D)
        if out.shape != shape:
            _shape(out, shape, name + "_out")
        if t.dtype is not one.dtype or out.dtype is not one.dtype:
            raise ValueError("q, k and their outputs must have one dtype")
        ptrs.append((_sptr(t, name, dev), _sptr(out, name + "_out", dev)))
        strides.append((t.stride()[:3], out.stride()[:3]))
        heads.append(shape[2])
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None and w.shape != (D,):
            _shape(w, (D,), name)
    rot, axes, turns, axis, pos = 0, 1, 0, 0, 0
    if rope is not None:
        rot, axes = rope.rot_dim, rope.num_axes
        if positions is None or (positions.shape != (axes, B, M)
                                 and (axes > 1 or positions.shape != (B, M))):
            raise ValueError("positions must be [%d, %d, %d]" % (axes, B, M))
        turns = _ptr(rope.turns, torch.int64, "the rotation's frequencies", dev)
        axis = _ptr(rope.axis, i32, "the rotation's axes", dev)
        pos = _ptr(positions, i32, "positions", dev)
    if count is not None and count.shape != (B,):
        _shape(count, (B,), "count")
    args = _NORM_ROPE_ARGS.pack(
        ptrs[0][0], ptrs[1][0], ptrs[0][1], ptrs[1][1], _dtype_code(one, "q and k", True), B, M,
        heads[0], heads[1], D, rot, 1 if rope is not None and rope.adjacent else 0, axes, eps,
        *strides[0][0], *strides[1][0], *strides[0][1], *strides[1][1],
        _ptr(q_weight, f32, "q_weight", dev), _ptr(k_weight, f32, "k_weight", dev), pos, turns,
        axis, _ptr(count, i32, "count", dev))
    _run("hs_norm_rope", dev, args, _raw_stream(stream, dev))


def bounds_shape(num_requests: int, max_seq_len: int, block_tokens: int, num_kv_heads: int,
                 head_dim: int):
    """Shape of the bounds on the keys of a store (hs_bound_keys)."""
    return (num_requests, -(-max_seq_len // block_tokens), num_kv_heads, 2, head_dim)


def _bounds(bounds, block_tokens, max_seq_len, heads, dim) -> int:
    """Requests of bounds [R, NB, Hkv, 2, D]."""
    if block_tokens < 1 or max_seq_len < 1:
        raise ValueError("need block_tokens >= 1 and max_seq_len >= 1")
    R = bounds.shape[0] if bounds.dim() else 0
    if bounds.shape != (R, -(-max_seq_len // block_tokens), heads, 2, dim):
        _shape(bounds, bounds_shape(R, max_seq_len, block_tokens, heads, dim), "bounds")
    return R


def hs_bound_keys(k, req, start, count, block_tokens: int, max_seq_len: int, bounds,
                  stream=None) -> None:
    """Least and greatest key of each block of tokens: k [batch, tokens, Hkv, D] (bf16 or fp16,
    any strides but a dense last dimension) are the tokens [start[b], start[b] + count[b]) of
    request req[b]; bounds [R, NB, Hkv, 2, D] of k's type, updated."""
    import torch
    B, M, H, D = _heads(k, "k")
    R = _bounds(bounds, block_tokens, max_seq_len, H, D)
    if bounds.dtype is not k.dtype:
        raise ValueError("bounds must have k's dtype")
    one = k.shape[:1]
    if req.shape != one or start.shape != one or count.shape != one:
        _shape(req, one, "req")
        _shape(start, one, "start")
        _shape(count, one, "count")
    i32, dev = torch.int32, _device_of(k, "k")
    _run("hs_bound_keys", dev, _sptr(k, "k", dev), _STRIDES.pack(*k.stride()[:3]),
         _dtype_code(k, "k", False), H, D, block_tokens, _ptr(req, i32, "req", dev),
         _ptr(start, i32, "start", dev), _ptr(count, i32, "count", dev), B, M,
         _ptr(bounds, bounds.dtype, "bounds", dev), R, max_seq_len, _raw_stream(stream, dev))


def hs_select_workspace_bytes(batch: int, steps: int, max_seq_len: int, block_tokens: int) -> int:
    """Device bytes of workspace that hs_select_blocks needs for these sizes."""
    n = load_library().hs_select_workspace_bytes(batch, steps, max_seq_len, block_tokens)
    if n == _NO_SIZES:
        raise HsError(HS_ERR_INVALID_ARG, "hs_select_workspace_bytes")
    return n


def hs_select_blocks(q, bounds, req, seq_lens, block_tokens: int, max_seq_len: int, first: int,
                     last: int, blocks, topk, scores, workspace, stream=None) -> None:
    """Selects key blocks for q [batch, steps, heads, D] (bf16 or fp16) by the bounds
    [R, NB, Hkv, 2, D] of the same type: the first `first`, the last `last` and those of the largest
    scores.  Outputs: blocks int32 [batch, steps, n] or None, topk int32
    [batch, steps, n * block_tokens] (their tokens), scores fp32 [batch, steps, NB]."""
    import torch
    B, S, H, D = _heads(q, "q")
    if bounds.dim() != 5:
        raise ValueError("bounds must be [requests, blocks, heads, 2, head_dim]")
    R = _bounds(bounds, block_tokens, max_seq_len, bounds.shape[2], D)
    if bounds.dtype is not q.dtype:
        raise ValueError("bounds must have q's dtype")
    if topk.dim() != 3 or topk.shape[2] % block_tokens:
        raise ValueError("topk must be [batch, steps, blocks * %d], got %s"
                         % (block_tokens, tuple(topk.shape)))
    n = topk.shape[2] // block_tokens
    one = q.shape[:1]
    if (topk.shape[:2] != q.shape[:2] or scores.shape != (B, S, bounds.shape[1])
            or req.shape != one or seq_lens.shape != one
            or (blocks is not None and blocks.shape != (B, S, n))):
        _shape(topk, (B, S, n * block_tokens), "topk")
        _shape(scores, (B, S, bounds.shape[1]), "scores")
        _shape(req, one, "req")
        _shape(seq_lens, one, "seq_lens")
        _shape(blocks, (B, S, n), "blocks")
    i32, dev = torch.int32, _device_of(q, "q")
    args = _SELECT_ARGS.pack(
        _sptr(q, "q", dev), _ptr(bounds, bounds.dtype, "bounds", dev), _dtype_code(q, "q", False),
        B, S, H, bounds.shape[2], D, R, max_seq_len, block_tokens, n, first, last,
        *q.stride()[:3], _ptr(req, i32, "req", dev), _ptr(seq_lens, i32, "seq_lens", dev),
        _ptr(blocks, i32, "blocks", dev), _ptr(topk, i32, "topk", dev),
        _ptr(scores, torch.float32, "scores", dev),
        _ptr(workspace, workspace.dtype, "workspace", dev),
        workspace.numel() * workspace.element_size())
    _run("hs_select_blocks", dev, args, _raw_stream(stream, dev))


def hs_prefix_workspace_bytes(fmt: HsKvFormat, batch: int, steps: int, num_heads: int,
                              num_prefixes: int) -> int:
    """Device bytes of workspace that hs_attend_prefix needs for these sizes."""
    args = _HsPrefixArgs(batch=batch, steps=steps, num_heads=num_heads, num_prefixes=num_prefixes)
    n = load_library().hs_prefix_workspace_bytes(fmt, ctypes.byref(args))
    if n == _NO_SIZES:
        raise HsError(HS_ERR_INVALID_ARG, "hs_prefix_workspace_bytes")
    return n


def hs_attend_prefix(fmt: HsKvFormat, q, rows, scales, prefix, lens, starts, out, lse=None,
                     join_out=None, join_lse=None, sm_scale: Optional[float] = None,
                     workspace=None, stream=None) -> None:
    """Attention of q [batch, steps, heads, D] (bf16 or fp16) over prefixes that consecutive batch
    rows share: rows starts[p] .. starts[p + 1] - 1 (starts int32 [P + 1]) attend to the first
    lens[p] tokens of request prefix[p] of the store rows uint8 [R, L, W] (device memory), scales fp32
    [R, NB, 2, Hkv].  Outputs: out as q, lse fp32 [batch, steps, heads].  join_out and join_lse: the
    same queries' attention over other tokens, to be joined (they may be out and lse).
    sm_scale: 1 / sqrt(D) by default."""
    import torch
    B, S, H, D = _heads(q, "q")
    if D != fmt.head_dim:
        raise ValueError("q must be [batch, steps, heads, %d], got %s"
                         % (fmt.head_dim, tuple(q.shape)))
    R, L = _store(fmt, rows, scales, "")
    P = prefix.shape[0] if prefix.dim() else 0
    if prefix.shape != (P,) or lens.shape != (P,) or starts.shape != (P + 1,):
        _shape(prefix, (P,), "prefix")
        _shape(lens, (P,), "lens")
        _shape(starts, (P + 1,), "starts")
    if out.shape != q.shape:
        _shape(out, q.shape, "out")
    if out.dtype is not q.dtype:
        raise ValueError("out must have q's dtype")
    if lse is not None and lse.shape != (B, S, H):
        _shape(lse, (B, S, H), "lse")
    dev, join, strides = _device_of(q, "q"), 0, (0, 0, 0)
    if (join_out is None) != (join_lse is None):
        raise ValueError("join_out and join_lse must be given together")
    if join_out is not None:
        if join_out.dtype is not q.dtype:
            raise ValueError("join_out must have q's dtype")
        _shape(join_out, q.shape, "join_out")
        _shape(join_lse, (B, S, H), "join_lse")
        join, strides = _sptr(join_out, "join_out", dev), join_out.stride()[:3]
    _device_of(rows, "rows")  # they are copied in tiles, which takes device memory
    i32, f32 = torch.int32, torch.float32
    args = _PREFIX_ARGS.pack(
        _sptr(q, "q", dev), _sptr(out, "out", dev), _dtype_code(q, "q", False), B, S, H, R, L, P,
        D ** -0.5 if sm_scale is None else sm_scale, *q.stride()[:3], *out.stride()[:3], *strides,
        _ptr(rows, torch.uint8, "rows", dev), _ptr(scales, f32, "scales", dev),
        _ptr(prefix, i32, "prefix", dev), _ptr(lens, i32, "lens", dev),
        _ptr(starts, i32, "starts", dev), _ptr(lse, f32, "lse", dev), join,
        _ptr(join_lse, f32, "join_lse", dev),
        0 if workspace is None else _ptr(workspace, workspace.dtype, "workspace", dev),
        0 if workspace is None else workspace.numel() * workspace.element_size())
    _run("hs_attend_prefix", dev, fmt, args, _raw_stream(stream, dev))
