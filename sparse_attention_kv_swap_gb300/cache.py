"""Memory plumbing around the C ABI: allocates the caller-owned buffers with
PyTorch (pinned host pools, device KV buffers, state, workspace) and forwards
each call to the library.  Nothing here computes any part of the swap-in."""
from __future__ import annotations

import contextlib
from typing import Dict, List, Optional

import torch

from . import binding as B


class SwapInCache:
    """One swap-in cache: pinned host pools + device hot buffers for all layers."""

    def __init__(self, cfg: B.HsConfig, host_pools: Optional[List[torch.Tensor]] = None,
                 device: Optional[torch.device] = None, stream=None):
        rc = B.hs_config_check(cfg)
        if rc != B.HS_OK:
            raise B.HsError(rc, "hs_config_check")
        self.cfg = cfg
        self.device = torch.device(device or "cuda")
        R, L, W = cfg.num_requests, cfg.max_seq_len, cfg.item_size_bytes
        self.H, self.C = cfg.hot_buffer_size, cfg.max_steps * cfg.top_k
        if host_pools is None:
            host_pools = [torch.empty((R, L, W), dtype=torch.uint8, pin_memory=True)
                          for _ in range(cfg.num_layers)]
        self.host_pools = host_pools
        self.E = cfg.extra_page_size
        rows = B.hs_device_kv_bytes(cfg) // W  # hot + scratch rows, then the extra pages
        self.device_kv = [torch.empty((rows, W), dtype=torch.uint8, device=self.device)
                          for _ in range(cfg.num_layers)]
        self.state = torch.empty(B.hs_state_bytes(cfg), dtype=torch.uint8, device=self.device)
        self.workspace = torch.empty(B.hs_workspace_bytes(cfg), dtype=torch.uint8,
                                     device=self.device)
        self.handle = B.hs_create_state(cfg, self.host_pools, self.device_kv, self.state,
                                        self.workspace, stream)

    @staticmethod
    def _allocate_on(stream):
        """Outputs that a call allocates belong to the stream it runs on: memory of another
        stream may still be in use there."""
        return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)

    def _workspace(self, o: Dict[str, torch.Tensor], name: str, need: int) -> None:
        """A workspace among a call's outputs; one kept from a smaller call gives way to a larger."""
        held = o.get(name)
        if held is None or held.numel() * held.element_size() < need:
            o[name] = torch.empty(need, dtype=torch.uint8, device=self.device)

    def swap_in(self, req_pool_indices: torch.Tensor, seq_lens: torch.Tensor,
                topk: torch.Tensor, layer_id: int = 0, stats: bool = False, plan: bool = False,
                out: Optional[Dict[str, torch.Tensor]] = None, stream=None):
        Bn, S, K = topk.shape
        o = dict(out or {})
        with self._allocate_on(stream):
            if "device_locs" not in o:
                o["device_locs"] = torch.empty((Bn, S, K), dtype=torch.int32, device=self.device)
            if stats and "stats" not in o:
                o["stats"] = torch.empty((Bn, B.HS_NUM_STATS), dtype=torch.int32, device=self.device)
            if plan and "miss_src" not in o:
                o["miss_src"] = torch.full((Bn, self.C), -1, dtype=torch.int64, device=self.device)
                o["miss_dst"] = torch.full((Bn, self.C), -1, dtype=torch.int64, device=self.device)
                o["miss_count"] = torch.empty(Bn, dtype=torch.int32, device=self.device)
        B.hs_swap_in(self.handle, req_pool_indices, seq_lens, topk, layer_id, o["device_locs"],
                     o.get("stats"), o.get("miss_src"), o.get("miss_dst"), o.get("miss_count"),
                     stream)
        return o

    def page_table(self, topk: torch.Tensor, seq_lens: torch.Tensor, page_size: int,
                   out: Optional[Dict[str, torch.Tensor]] = None, stream=None):
        Bn, S, K = topk.shape
        o = dict(out or {})
        with self._allocate_on(stream):
            o.setdefault("pages", torch.empty((Bn, S * K), dtype=torch.int32, device=self.device))
            o.setdefault("num_pages", torch.empty(Bn, dtype=torch.int32, device=self.device))
            o.setdefault("token_page", torch.empty((Bn, S, K), dtype=torch.int32, device=self.device))
        B.hs_page_table(topk, seq_lens, self.cfg.max_seq_len, page_size, o["pages"],
                        o["num_pages"], o["token_page"], stream)
        return o

    def append_rows(self, req: torch.Tensor, tok: torch.Tensor, seq_lens: torch.Tensor,
                    rows: torch.Tensor, layer_id: int = 0, stream=None) -> None:
        """Write-back of newly decoded KV rows (host pool, extra page, hot copy)."""
        B.hs_append_rows(self.handle, layer_id, req, tok, seq_lens, rows, stream)

    # ---- 8-bit key/value rows (binding.make_kv_format) --------------------------

    def kv_scales(self, fmt: B.HsKvFormat) -> torch.Tensor:
        """Scales of one layer's rows: fp32 [R, NB, 2, Hkv]."""
        return torch.zeros(fmt.scales_shape(self.cfg.num_requests, self.cfg.max_seq_len),
                           device=self.device)

    def append_kv(self, fmt: B.HsKvFormat, scales: torch.Tensor, k: torch.Tensor,
                  v: torch.Tensor, req: torch.Tensor, start: torch.Tensor, count: torch.Tensor,
                  layer_id: int = 0, stream=None) -> None:
        """Quantises new keys and values [batch, tokens, Hkv, D] and writes them back
        (host pool, extra page, hot copy)."""
        B.hs_append_kv(self.handle, layer_id, fmt, k, v, req, start, count, scales, stream)

    def attend(self, fmt: B.HsKvFormat, scales: torch.Tensor, q: torch.Tensor,
               topk: torch.Tensor, device_locs: torch.Tensor, req_pool_indices: torch.Tensor,
               layer_id: int = 0, lse: bool = False, weights: bool = False,
               acc: Optional[torch.Tensor] = None, sm_scale: Optional[float] = None,
               out: Optional[Dict[str, torch.Tensor]] = None, stream=None):
        """Attention of q [batch, steps, heads, D] over the rows that a swap-in located."""
        if not 0 <= layer_id < self.cfg.num_layers:  # a list would take -1 for its last entry
            raise B.HsError(B.HS_ERR_INVALID_ARG, "SwapInCache.attend")
        Bn, S, K = topk.shape
        o = dict(out or {})
        with self._allocate_on(stream):
            if "out" not in o:
                o["out"] = torch.empty(q.shape, dtype=q.dtype, device=self.device)
            if lse and "lse" not in o:
                o["lse"] = torch.empty(q.shape[:3], device=self.device)
            if (weights or (acc is not None and S > 1)) and "weights" not in o:
                o["weights"] = torch.empty((Bn, S, K), device=self.device)
            need = B.hs_attend_workspace_bytes(fmt, Bn, S, K, q.shape[2])
            if need:
                self._workspace(o, "workspace", need)
        B.hs_attend(fmt, q, self.device_kv[layer_id], device_locs, topk, req_pool_indices, scales,
                    self.cfg.max_seq_len, o["out"], o.get("lse"), o.get("weights"), acc, sm_scale,
                    o.get("workspace"), stream)
        return o

    # ---- selection by bounds on the keys, shared prefixes -----------------------

    def key_bounds(self, fmt: B.HsKvFormat, dtype: torch.dtype, block_tokens: int) -> torch.Tensor:
        """Bounds on one layer's keys, which are of `dtype`: [R, NB, Hkv, 2, D]."""
        return torch.zeros(B.bounds_shape(self.cfg.num_requests, self.cfg.max_seq_len, block_tokens,
                                          fmt.num_kv_heads, fmt.head_dim), dtype=dtype,
                           device=self.device)

    def bound_keys(self, bounds: torch.Tensor, block_tokens: int, k: torch.Tensor,
                   req: torch.Tensor, start: torch.Tensor, count: torch.Tensor,
                   stream=None) -> None:
        """Brings new keys [batch, tokens, Hkv, D], those of append_kv, into their blocks' bounds.
        (evict moves keys to other blocks, and makes the bounds that it is given anew.)"""
        B.hs_bound_keys(k, req, start, count, block_tokens, self.cfg.max_seq_len, bounds, stream)

    def select_blocks(self, bounds: torch.Tensor, block_tokens: int, q: torch.Tensor,
                      req_pool_indices: torch.Tensor, seq_lens: torch.Tensor, first: int = 1,
                      last: int = 1, out: Optional[Dict[str, torch.Tensor]] = None, stream=None):
        """The top-k tokens for swap_in, as whole blocks, for q [batch, steps, heads, D]: the first
        `first` blocks, the last `last` and those of the largest bounds on their scores."""
        if block_tokens < 1 or self.cfg.top_k % block_tokens:
            raise ValueError("the cache's top_k (%d) must be a multiple of block_tokens (%d)"
                             % (self.cfg.top_k, block_tokens))
        Bn, S = q.shape[:2]
        o = dict(out or {})
        with self._allocate_on(stream):
            if "topk" not in o:
                o["topk"] = torch.empty((Bn, S, self.cfg.top_k), dtype=torch.int32,
                                        device=self.device)
            if "scores" not in o:
                o["scores"] = torch.empty((Bn, S, bounds.shape[1]), device=self.device)
            self._workspace(o, "select_workspace", B.hs_select_workspace_bytes(
                Bn, S, self.cfg.max_seq_len, block_tokens))
        B.hs_select_blocks(q, bounds, req_pool_indices, seq_lens, block_tokens,
                           self.cfg.max_seq_len, first, last, o.get("blocks"), o["topk"],
                           o["scores"], o["select_workspace"], stream)
        return o

    def attend_prefix(self, fmt: B.HsKvFormat, rows: torch.Tensor, scales: torch.Tensor,
                      q: torch.Tensor, prefix: torch.Tensor, lens: torch.Tensor,
                      starts: torch.Tensor, join: Optional[Dict[str, torch.Tensor]] = None,
                      sm_scale: Optional[float] = None,
                      out: Optional[Dict[str, torch.Tensor]] = None, stream=None):
        """Attention of q over prefixes that consecutive batch rows share, kept in device memory
        (rows [P, tokens, W] and their scales, as hs_quantize_kv writes them); join: what attend
        returned for the same q with lse=True, which is joined in (and may be `out` too)."""
        Bn, S, heads = q.shape[:3]
        o = dict(out or {})
        with self._allocate_on(stream):
            if "out" not in o:
                o["out"] = torch.empty(q.shape, dtype=q.dtype, device=self.device)
            if "lse" not in o:
                o["lse"] = torch.empty(q.shape[:3], device=self.device)
            self._workspace(o, "prefix_workspace", B.hs_prefix_workspace_bytes(
                fmt, Bn, S, heads, prefix.shape[0]))
        B.hs_attend_prefix(fmt, q, rows, scales, prefix, lens, starts, o["out"], o["lse"],
                           None if join is None else join["out"],
                           None if join is None else join["lse"], sm_scale,
                           o["prefix_workspace"], stream)
        return o

    def evict(self, fmt: B.HsKvFormat, scales: List[torch.Tensor], acc: List[torch.Tensor],
              requests: List[int], seq_lens: List[int], budget: int, recent: int,
              stream=None, bounds: Optional[List[torch.Tensor]] = None,
              block_tokens: Optional[int] = None) -> List[int]:
        """Cuts the given requests (lengths seq_lens) to `budget` tokens in every layer:
        the last `recent` and those of the largest accumulated weight acc[layer]
        [R, max_seq_len].  Kept rows move to the first positions of the host pools;
        scales[layer] and acc[layer] follow; the requests' cache state is reset and
        their new lengths are returned.  Bytes of a row past its keys and values move with it
        (the call then waits for the stream in every layer).  Needs budget rows of device
        memory per request.
        Kept keys move to other blocks: bounds[layer] (key_bounds, in blocks of block_tokens) are
        made anew for the requests, of the kept keys as attend reads them (code * scale, rounded to
        the bounds' type).  Without `bounds`, bounds that were kept up for them are stale.
        Arguments that do not fit the cache raise ValueError before anything changes."""
        self._check_evict(fmt, scales, acc, requests, seq_lens, budget, recent, bounds, block_tokens)
        if not requests:
            return []
        kept = [min(n, budget) for n in seq_lens]
        nb = fmt.num_blocks(budget)
        used = 2 * fmt.num_kv_heads * fmt.head_dim
        owner = torch.tensor(requests)[:, None]
        ctx = torch.cuda.stream(stream) if stream is not None else torch.cuda.stream(
            torch.cuda.current_stream(self.device))
        with torch.cuda.device(self.device), ctx:
            i32 = dict(dtype=torch.int32, device=self.device)
            req, lens = torch.tensor(requests, **i32), torch.tensor(seq_lens, **i32)
            at = torch.arange(len(requests), **i32)
            # the entries (request, position) that are written back
            each = torch.tensor(kept, device=self.device)
            total = sum(kept)
            row = torch.repeat_interleave(at.long(), each, output_size=total)
            pos = torch.arange(total, device=self.device) - (each.cumsum(0) - each)[row]
            keep = torch.empty((len(requests), budget), **i32)
            count = torch.empty(len(requests), **i32)
            sums = torch.empty((len(requests), budget), device=self.device)
            rows = torch.empty((len(requests), budget, self.cfg.item_size_bytes),
                               dtype=torch.uint8, device=self.device)
            self.reset_requests(req)
            for layer, pool in enumerate(self.host_pools):
                B.hs_evict(acc[layer], req, lens, recent, keep, count, sums)
                new = torch.zeros((len(requests), nb, 2, fmt.num_kv_heads), device=self.device)
                B.hs_compact_kv(fmt, pool, scales[layer], req, keep, count, rows, new, at,
                                handle=self.handle)
                if used < self.cfg.item_size_bytes:  # on the host, which has the pool at hand
                    index = keep.cpu().clamp_(min=0).long()
                    rows[..., used:] = pool[owner, index, used:].to(self.device)
                self.append_rows(req[row], pos.to(torch.int32), count[row], rows[row, pos], layer)
                scales[layer][req.long(), :nb] = new[:, :scales[layer].shape[1]]
                acc[layer][req.long()] = 0
                acc[layer][req.long(), :budget] = sums[:, :self.cfg.max_seq_len]
                for i in range(len(requests) if bounds is not None else 0):
                    k = self._keys(fmt, rows[i], new[i], bounds[layer].dtype)
                    self.bound_keys(bounds[layer], block_tokens, k[None], req[i:i + 1],
                                    torch.zeros_like(req[i:i + 1]), count[i:i + 1])
        return kept

    @staticmethod
    def _keys(fmt, rows, scales, dtype) -> torch.Tensor:
        """The keys [tokens, Hkv, D] that rows [tokens, W] hold, within the type's range."""
        shape = (rows.shape[0], fmt.num_kv_heads, fmt.head_dim)
        kind = torch.int8 if fmt.code == B.HS_KV_INT8 else torch.float8_e4m3fn
        codes = rows[:, :shape[1] * shape[2]].contiguous().view(kind).view(shape).float()
        each = scales[:, 0].repeat_interleave(fmt.block_tokens, 0)[:shape[0], :, None]
        most = torch.finfo(dtype).max
        return (codes * each).clamp_(-most, most).to(dtype)

    def _check_evict(self, fmt, scales, acc, requests, seq_lens, budget, recent, bounds=None,
                     block_tokens=None) -> None:
        """The arguments of evict, on the host: layers are cut one after the other, and indexing
        by a request knows no range, so nothing may be refused once the first kernel runs."""
        cfg = self.cfg
        R, L = cfg.num_requests, cfg.max_seq_len
        if not 0 <= recent <= budget or budget < 1:
            raise ValueError("need 0 <= recent <= budget and budget >= 1")
        if len(requests) != len(seq_lens) or any(not 0 <= n <= L for n in seq_lens):
            raise ValueError("need a length from 0 to %d for every request" % L)
        if any(not 0 <= q < R for q in requests) or len(set(requests)) != len(requests):
            raise ValueError("requests must be distinct and from 0 to %d" % (R - 1))
        rc = B.load_library().hs_kv_format_check(fmt)
        if rc != B.HS_OK or fmt.item_size_bytes != cfg.item_size_bytes:
            raise ValueError("the format must be valid and its rows %d bytes wide"
                             % cfg.item_size_bytes)
        if any(p.shape != (R, L, cfg.item_size_bytes) or p.dtype != torch.uint8
               for p in self.host_pools):
            raise ValueError("the host pools must be uint8 [%d, %d, %d]"
                             % (R, L, cfg.item_size_bytes))
        if (bounds is None) != (block_tokens is None):
            raise ValueError("bounds and block_tokens must be given together")
        if bounds is not None:
            if not 1 <= block_tokens <= B.HS_MAX_KV_BLOCK:
                raise ValueError("block_tokens must be from 1 to %d" % B.HS_MAX_KV_BLOCK)
            shape = B.bounds_shape(R, L, block_tokens, fmt.num_kv_heads, fmt.head_dim)
            if len(bounds) != cfg.num_layers or any(
                    t.shape != shape or t.dtype not in (torch.bfloat16, torch.float16)
                    or not t.is_contiguous() or t.device != self.device_kv[0].device
                    for t in bounds):
                raise ValueError("bounds must hold a contiguous bfloat16 or float16 tensor %s for "
                                 "each of the %d layers, on the cache's device"
                                 % (shape, cfg.num_layers))
        for name, given, shape in (("scales", scales, fmt.scales_shape(R, L)),
                                   ("acc", acc, (R, L))):
            if len(given) != cfg.num_layers or any(
                    t.shape != shape or t.dtype != torch.float32 or not t.is_contiguous()
                    or t.device != self.device_kv[0].device for t in given):
                raise ValueError("%s must hold a contiguous float32 tensor %s for each of the %d "
                                 "layers, on the cache's device" % (name, tuple(shape),
                                                                    cfg.num_layers))

    def reset_requests(self, req_pool_indices: torch.Tensor, stream=None) -> None:
        B.hs_reset_requests(self.handle, req_pool_indices, stream)

    def totals(self, layer_id: int = 0, reset: bool = False, stream=None):
        """Running sums of the per-request counters of one layer (HS_STAT_* order)."""
        return B.hs_get_stats(self.handle, layer_id, reset, stream)

    def status(self, stream=None):
        return B.hs_get_status(self.handle, stream)

    def export_request_state(self, layer_id: int, request: int, stream=None):
        return B.hs_export_request_state(self.handle, layer_id, request, stream)

    def close(self) -> None:
        self.handle.close()
