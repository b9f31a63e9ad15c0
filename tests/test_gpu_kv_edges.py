"""The 8-bit key/value row calls where they could go wrong, on the GPU."""
import numpy as np
import pytest
import torch

import kv_reference as ref
import sparse_attention_kv_swap_gb300 as pkg
from sparse_attention_kv_swap_gb300 import binding as B
from test_gpu_kv_rows import dev
from test_kv_edges import evict_refusals

pytestmark = pytest.mark.gpu


def test_cache_evict_refusals_change_nothing():
    """Whatever evict refuses, pools, scales, sums and the resident tokens of every layer stay."""
    from sparse_attention_kv_swap_gb300.cache import SwapInCache
    cache = SwapInCache(pkg.make_config(3, 40, 256, 16, 8, 1, num_layers=2))
    every = dev(np.arange(3, dtype=np.int32))
    lens = torch.full_like(every, 40)
    topk = dev(np.arange(8, dtype=np.int32)[None, None].repeat(3, 0))
    for layer, pool in enumerate(cache.host_pools):
        pool.random_(0, 120)
        cache.swap_in(every, lens, topk, layer)
    pools = [p.clone() for p in cache.host_pools]
    for kw in evict_refusals(lambda shape: torch.full(shape, 3.0, device="cuda")):
        with pytest.raises(ValueError):
            cache.evict(**kw)
        torch.cuda.synchronize()
        for t in kw["scales"] + kw["acc"]:
            assert (t == 3).all()
        for p, q in zip(cache.host_pools, pools):
            assert torch.equal(p, q)
    for layer in range(2):
        stats = cache.swap_in(every, lens, topk, layer, stats=True)["stats"]
        assert (stats[:, 0] == 8).all() and (stats[:, 3] == 0).all()  # hits, no misses
    assert cache.status() == (B.HS_OK, 0)
    cache.close()


class Evicted:
    """A cache whose requests are cut, next to the plain implementation's pools, scales and sums.
    W: the rows' width; the bytes past keys and values are the user's own."""

    def __init__(self, rng, pools=None, R=3, L=90, layers=2, heads=2, D=64, T=16, W=256):
        from sparse_attention_kv_swap_gb300.cache import SwapInCache
        self.fmt = pkg.make_kv_format(heads, D, T, B.HS_KV_E4M3, W)
        self.cache = SwapInCache(pkg.make_config(R, L, W, 40, 30, 1, num_layers=layers,
                                                 extra_page_size=16), pools)
        self.scales = [self.cache.kv_scales(self.fmt) for _ in range(layers)]
        self.acc = [dev(rng.random((R, L)).astype(np.float32)) for _ in range(layers)]
        every = torch.arange(R, dtype=torch.int32, device="cuda")
        for l, pool in enumerate(self.cache.host_pools):
            pool.random_(0, 120)
            kv = torch.from_numpy(rng.standard_normal((2, R, L, heads, D))).bfloat16()
            self.cache.append_kv(self.fmt, self.scales[l], dev(kv[0]), dev(kv[1]), every,
                                 torch.zeros_like(every), torch.full_like(every, L), layer_id=l)
        torch.cuda.synchronize()

    def check(self, requests, lens, budget, recent, evict=None):
        """evict(), and every layer's pool, scales and sums against the plain implementation."""
        fmt, cache = self.fmt, self.cache
        heads, D, T, W = fmt.num_kv_heads, fmt.head_dim, fmt.block_tokens, fmt.item_size_bytes
        was = [(p.clone(), s.cpu(), a.cpu().numpy())
               for p, s, a in zip(cache.host_pools, self.scales, self.acc)]
        got = (evict or cache.evict)(fmt, self.scales, self.acc, requests, lens, budget, recent)
        torch.cuda.synchronize()
        assert got == [min(n, budget) for n in lens]
        for l, (pool, scale, acc) in enumerate(was):
            keep, kept, ka = ref.evict(acc, requests, lens, recent, budget)
            n = len(requests)
            dst = torch.zeros((n, budget, W), dtype=torch.uint8)
            ds = torch.zeros(fmt.scales_shape(n, budget))
            ref.compact(pool, scale, requests, torch.from_numpy(keep), torch.from_numpy(kept), dst,
                        ds, list(range(n)), T, heads, D, "e4m3")
            for i, q in enumerate(requests):
                m = int(kept[i])  # the user's bytes stay with their token
                dst[i, :m, 2 * heads * D:] = pool[q, torch.from_numpy(keep[i, :m]).long(),
                                                  2 * heads * D:]
                pool[q, :m] = dst[i, :m]
                blocks = -(-m // T)
                assert torch.equal(self.scales[l][q, :blocks].cpu(), ds[i, :blocks])
                acc[q], acc[q, :budget] = 0, ka[i, :acc.shape[1]]
            assert torch.equal(cache.host_pools[l], pool)
            assert np.array_equal(self.acc[l].cpu().numpy(), acc)
        assert cache.status() == (B.HS_OK, 0)


def test_cache_evict_from_pageable_pools():
    """Pools of pageable memory, where the device reads them, are cut like pinned ones."""
    rng = np.random.default_rng(41)
    pools = [torch.empty((3, 90, 256), dtype=torch.uint8) for _ in range(2)]
    assert not pools[0].is_pinned()
    try:
        e = Evicted(rng, pools)
    except pkg.HsError as error:
        assert error.code == B.HS_ERR_INVALID_ARG
        return
    e.check([2, 0], [90, 37], 40, 7)
    e.cache.close()


@pytest.mark.parametrize("W", [272, 400])
def test_cache_evict_moves_the_whole_row(W):
    """Rows wider than their keys and values: the other bytes stay with their token."""
    e = Evicted(np.random.default_rng(W), W=W)
    e.check([1, 2, 0], [90, 61, 12], 33, 4)
    e.check([2], [33], 20, 0)
    e.cache.close()
