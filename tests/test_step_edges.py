"""Calls around a decode step on the CPU, at the edges of what they accept."""
import ctypes

import pytest
import torch

import sparse_attention_kv_swap_gb300 as pkg
from sparse_attention_kv_swap_gb300 import binding as B


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_kv_swap_gb300 import build
    build.build()
    return B.load_library()


@pytest.mark.parametrize("batch,steps,heads", [
    (2 ** 31 - 1, 1, 1), (2 ** 31 - 256, 1, 1), (1, 2 ** 31 - 1, 1), (2 ** 24, 1, 128),
    (2 ** 31 - 1, 2 ** 31 - 1, 128), (2 ** 30, 2 ** 28, 64)])  # products beyond 63 bits
def test_attend_prefix_refuses_rows_beyond_32_bits(lib, batch, steps, heads):
    """With the rows that a last tile lacks, and whatever their product overflows to."""
    fmt = pkg.make_kv_format(1, 32, 16)
    args = B._HsPrefixArgs(q_dev=0x20000, out_dev=0x20000, dtype=B.HS_DTYPE_BF16, batch=batch,
                           steps=steps, num_heads=heads, num_requests=1, max_seq_len=64,
                           num_prefixes=0)
    call = lib.hs_attend_prefix(ctypes.byref(fmt), ctypes.byref(args), None)
    assert call == B.HS_ERR_UNSUPPORTED
    with pytest.raises(pkg.HsError):
        pkg.hs_prefix_workspace_bytes(fmt, batch, steps, heads, 1)


def test_prefix_workspace_of_many_rows(lib):
    fmt = pkg.make_kv_format(1, 32, 16)
    assert pkg.hs_prefix_workspace_bytes(fmt, 2 ** 31 - 4097, 1, 1, 1) > 0


def test_cache_workspaces_grow(lib, monkeypatch):
    """Outputs that were used for a smaller call, or for none, serve a larger one."""
    from sparse_attention_kv_swap_gb300 import cache as C
    cache = C.SwapInCache.__new__(C.SwapInCache)  # the sizes alone are looked at
    cache.cfg, cache.device = pkg.make_config(4, 4096, 256, 48, 48, 1), torch.device("cpu")
    cache.device_kv = [torch.empty(0)]
    fmt, wide = pkg.make_kv_format(2, 64, 16), pkg.make_kv_format(2, 256, 16)
    given = []
    for name, at in (("hs_select_blocks", 11), ("hs_attend_prefix", 12), ("hs_attend", 13)):
        monkeypatch.setattr(B, name, lambda *a, at=at: given.append(a[at]))
    bounds = cache.key_bounds(fmt, torch.bfloat16, 16)
    one = torch.zeros(64, dtype=torch.int32)

    def q(batch, dim=64):
        return torch.zeros((batch, 1, 128, dim), dtype=torch.bfloat16)

    def select(batch, out):
        out = {x: y for x, y in out.items() if x == "select_workspace"}
        return cache.select_blocks(bounds, 16, q(batch), one, one, out=out)

    o = select(0, {})
    for batch in (1, 64, 2):
        held = o["select_workspace"]
        o = select(batch, o)
        need = pkg.hs_select_workspace_bytes(batch, 1, 4096, 16)
        assert given[-1] is o["select_workspace"] and given[-1].numel() >= need
    assert held is o["select_workspace"]

    def prefix(f, batch, out):
        rows = torch.empty((1, 4, f.item_size_bytes), dtype=torch.uint8)
        out = {x: y for x, y in out.items() if x == "prefix_workspace"}
        return cache.attend_prefix(f, rows, rows, q(batch, f.head_dim), one[:1], one, one, out=out)

    o = prefix(fmt, 0, {})
    for f, batch in ((fmt, 2), (wide, 2), (fmt, 1)):
        held = o["prefix_workspace"]
        o = prefix(f, batch, o)
        need = pkg.hs_prefix_workspace_bytes(f, batch, 1, 128, 1)
        assert given[-1] is o["prefix_workspace"] and given[-1].numel() >= need
    assert held is o["prefix_workspace"]

    def attend(batch, K, out):
        topk = torch.zeros((batch, 1, K), dtype=torch.int32)
        return cache.attend(fmt, one, q(batch), topk, topk, one, out=out)

    sizes = [pkg.hs_attend_workspace_bytes(fmt, b, 1, 32768, 128) for b in (1, 2)]
    assert 0 < sizes[0] < sizes[1]
    o = {"workspace": attend(1, 32768, {})["workspace"]}
    assert given[-1].numel() == sizes[0]
    o = attend(2, 32768, o)
    assert given[-1] is o["workspace"] and given[-1].numel() == sizes[1]
    assert "workspace" not in attend(1, 16, {})


def test_cache_evict_refuses_bounds(lib):
    """Bounds that do not fit the cache are refused before anything changes."""
    from test_kv_edges import cpu_cache
    cache = cpu_cache()  # 3 requests of 40 tokens in 2 layers
    fmt = pkg.make_kv_format(2, 64, 16)
    scales, acc = [torch.ones((3, 3, 2, 2))] * 2, [torch.ones((3, 40))] * 2

    def bounds(*shape, dtype=torch.bfloat16, n=2):
        return [torch.zeros(shape, dtype=dtype) for _ in range(n)]

    for b, T in ((bounds(3, 5, 2, 2, 64), None), (None, 8), (bounds(3, 5, 2, 2, 64), 0),
                 (bounds(3, 5, 2, 2, 64), -8), (bounds(3, 5, 2, 2, 64), 16),
                 (bounds(3, 1, 2, 2, 64), 4097), (bounds(2, 5, 2, 2, 64), 8),
                 (bounds(3, 5, 2, 2, 64, n=1), 8), (bounds(3, 5, 2, 2, 64, n=3), 8),
                 (bounds(3, 5, 2, 2, 64, dtype=torch.float32), 8),
                 ([x.transpose(0, 1) for x in bounds(5, 3, 2, 2, 64)], 8),
                 (bounds(3, 5, 2, 2, 64, n=1) + bounds(3, 5, 1, 2, 64, n=1), 8)):
        with pytest.raises(ValueError, match="bounds|block_tokens"):
            cache.evict(fmt, scales, acc, [0], [40], 8, 2, bounds=b, block_tokens=T)
