"""The 8-bit key/value row calls where they could go wrong, on the GPU."""
import numpy as np
import pytest
import torch

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
