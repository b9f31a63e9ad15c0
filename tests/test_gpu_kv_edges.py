"""The 8-bit key/value row calls where they could go wrong, on the GPU."""
import numpy as np
import pytest
import torch

import kv_reference as ref
import sparse_attention_kv_swap_gb300 as pkg
from sparse_attention_kv_swap_gb300 import binding as B
from test_gpu_kv_rows import Attend, dev, random_codes
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


# ---- attention: V scales far apart ----------------------------------------------

@pytest.mark.parametrize("light", [True, False], ids=["quiet", "even"])
@pytest.mark.parametrize("gap", [12, 16, 20, 24, 30, 60, 90])
@pytest.mark.parametrize("heads,G,D,K,code", [(2, 4, 128, 300, "e4m3"), (1, 16, 64, 1000, "int8"),
                                              (2, 6, 256, 90, "int8"), (1, 8, 192, 60, "e4m3")])
def test_attend_v_scales_far_apart(heads, G, D, K, code, gap, light):
    """A block in five has V scales 2^gap times the others', on tokens whose weight makes up for
    the scale, or for e^20 times that.  Bound: as for any scales, with f16's smallest step
    counted from the largest product of weight and V scale: 2^-25 of 2^14.5 for every entry."""
    rng = np.random.default_rng(gap + D)
    a = Attend(rng, 2, 1, K, heads, G, D, 4, code, "bf16")
    used = np.unique(a.locs[a.locs >= 0])
    loud = (a.topk // a.T) % 5 == 0
    a.scales[:, :, 1] *= 2.0 ** -gap
    a.scales[:, ::5, 1] *= 2.0 ** gap
    # channel 0 of K alone carries the gap in the scores
    a.q[..., 0] = 1
    a.rows[used[:, None], np.arange(heads)[None] * D] = 0
    one = {"e4m3": 0x70, "int8": 64}[code]  # 128 (e4m3), 64
    value = {"e4m3": 128.0, "int8": 64.0}[code]
    for b in range(2):
        at = a.locs[b, 0][loud[b, 0] & (a.locs[b, 0] >= 0)]
        a.rows[at[:, None], np.arange(heads)[None] * D] = one
    a.scales[:, :, 0] = 2.0 ** -7
    down = -(gap * np.log(2.0) + (20.0 if light else 0.0))
    a.q[..., 0] = float(np.float32(down / (value * 2.0 ** -7 * a.sm_scale)))
    want = a.reference()
    out = a.run()[0].cpu().double().numpy()
    assert np.isfinite(out).all()
    x = ref.decode_table(code)[a.rows[..., :2 * heads * D]].reshape(a.N, 2, heads, D)
    u = torch.finfo(torch.bfloat16).eps / 2
    dz = (D + 8) * 2.0 ** -23 * want["logit"] + 2.0 ** -20 + K * 2.0 ** -24
    for b in range(2):
        ok = a.locs[b, 0] >= 0
        k = x[a.locs[b, 0, ok], 0] * a.scales[a.req[b], a.topk[b, 0, ok] // 4, 0][..., None]
        v = a.scales[a.req[b], a.topk[b, 0, ok] // 4, 1].astype(np.float64)
        for i in range(heads * G):
            z = (k[:, i // G] @ a.q.double().numpy()[b, 0, i]) * a.sm_scale
            most = (np.exp(z - want["lse"][b, 0, i]) * v[:, i // G]).max()
            tol = (u * np.abs(want["out"][b, 0, i])
                   + want["spread"][b, 0, i] * (2.0 ** -11 + 2 * dz[b, 0, i]) * (1 + u)
                   + K * 2.0 ** -39 * most * 448 + 1e-37)
            err = np.abs(out[b, 0, i] - want["out"][b, 0, i])
            assert (err <= tol).all(), (b, i, (err / tol).max())


@pytest.mark.parametrize("exponent", [-140, -126, -110, 100, 120])
def test_attend_v_scales_of_any_size(exponent):
    """V scales near either end of 32 bits, the codes so small or large that the output is in
    range."""
    rng = np.random.default_rng(200 + exponent)
    a = Attend(rng, 2, 1, 120, 2, 4, 64, 8, "e4m3", "bf16")
    a.scales[:, :, 1] = 2.0 ** exponent
    if exponent > 0:  # V codes 2^-9 .. 2^-6
        used = np.unique(a.locs[a.locs >= 0])
        a.rows[used, 128:256] = rng.integers(1, 9, (used.size, 128))
    want = a.reference()
    out = a.run()[0].cpu().double().numpy()
    u = torch.finfo(torch.bfloat16).eps / 2
    dz = (64 + 8) * 2.0 ** -23 * want["logit"] + 2.0 ** -20 + 120 * 2.0 ** -24
    tol = (u * np.abs(want["out"]) + want["spread"] * (2.0 ** -11 + 2 * dz[..., None]) * (1 + u)
           + 120 * 2.0 ** -39 * 2.0 ** exponent * 448 + 2.0 ** -134)
    err = np.abs(out - want["out"])
    assert (err <= tol).all(), (err / tol).max()


# ---- attention: many wide heads ---------------------------------------------------

@pytest.mark.parametrize("heads,G,D,K,code", [(32, 4, 192, 64, "e4m3"), (64, 2, 192, 130, "int8"),
                                              (96, 1, 192, 40, "e4m3"), (128, 1, 192, 300, "e4m3"),
                                              (14, 9, 192, 0, "e4m3"), (40, 3, 256, 90, "int8"),
                                              (128, 1, 256, 64, "e4m3"), (112, 1, 256, 1, "int8"),
                                              (8, 16, 256, 8192, "e4m3"), (1, 128, 256, 8192, "int8"),
                                              (16, 8, 256, 5000, "e4m3")])
def test_attend_many_wide_heads(heads, G, D, K, code):
    """Head layouts whose outputs leave room for fewer warps than usual."""
    rng = np.random.default_rng(heads + D + K)
    a = Attend(rng, 2 if K < 1000 else 1, 2 if K < 100 else 1, K, heads, G, D, 16, code, "bf16")
    B_, S = a.topk.shape[:2]
    n = pkg.hs_attend_workspace_bytes(a.fmt, B_, S, K, heads * G)
    ws = torch.full((n,), 0xff, dtype=torch.uint8, device="cuda") if n else None
    a.check(a.run(workspace=ws))


# ---- streams ------------------------------------------------------------------------

def test_outputs_belong_to_the_stream_of_the_call():
    """While the current stream has work pending, calls on another stream allocate their
    outputs: neither may they take memory that the pending work still reads, nor may
    the current stream write them."""
    from sparse_attention_kv_swap_gb300.cache import SwapInCache
    rng = np.random.default_rng(51)
    Bn, K, heads, D, L = 64, 64, 32, 128, 200
    cache = SwapInCache(pkg.make_config(Bn, L, 2 * D, 2 * K, K, 1))
    cache.host_pools[0].random_(0, 120)
    fmt = pkg.make_kv_format(1, D, 16)
    scales = cache.kv_scales(fmt) + 2.0 ** -7
    req = torch.arange(Bn, dtype=torch.int32, device="cuda")
    lens = torch.full_like(req, L)
    topk = dev(np.stack([rng.permutation(L)[:K] for _ in range(Bn)]).astype(np.int32)[:, None])
    q = dev(torch.from_numpy(rng.standard_normal((Bn, 1, heads, D))).bfloat16())
    want_plan = cache.swap_in(req, lens, topk, plan=True)
    want = cache.attend(fmt, scales, q, topk, want_plan["device_locs"], req, lse=True,
                        weights=True)
    cache.reset_requests(req)
    side = torch.cuda.Stream()
    like = [want[k] for k in ("out", "lse", "weights")] + [
        want_plan[k] for k in ("device_locs", "miss_src", "miss_dst", "miss_count")]
    old = [torch.full_like(t, 7) for t in like]
    new = [torch.empty_like(t) for t in like]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # some 50 ms of the current stream
    for x, y in zip(old, new):
        y.copy_(x)
    del x, y
    old.clear()  # free for the current stream, behind its copies
    plan = cache.swap_in(req, lens, topk, plan=True, stream=side)
    got = cache.attend(fmt, scales, q, topk, plan["device_locs"], req, lse=True, weights=True,
                       stream=side)
    torch.cuda.synchronize()
    assert all((y == 7).all() for y in new)
    for k, x in list(want.items()) + list(want_plan.items()):
        assert torch.equal(got[k] if k in got else plan[k], x), k
    cache.close()


# ---- attention: queries of one large element ------------------------------------------

@pytest.mark.parametrize("gap", [12, 20, 28, 34, 45])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_attend_small_query_elements(gap, code):
    """One element of the query 2^gap times the others, on a channel whose K codes are zero: the
    others' products stay exact to 2^-39 of the largest element."""
    rng = np.random.default_rng(300 + gap)
    heads, G, D, K = 2, 4, 64, 200
    a = Attend(rng, 2, 1, K, heads, G, D, 8, code, "bf16")
    a.sm_scale = 2.0 ** gap * D ** -0.5
    q = a.q.double() * 2.0 ** -gap
    q[..., 5] = 1
    a.q = q.to(torch.bfloat16)
    used = np.unique(a.locs[a.locs >= 0])
    a.rows[used[:, None], np.arange(heads)[None] * D + 5] = 0
    want = a.reference()
    out, lse, _ = (x.cpu().double().numpy() for x in a.run())
    # a score's error: 32-bit sums as in Attend.check, and every query element's own
    size = a.scales[:, :, 0].max() * {"e4m3": 448, "int8": 127}[code]
    dz = ((D + 8) * 2.0 ** -23 * want["logit"] + 2.0 ** -20 + K * 2.0 ** -24
          + D * 2.0 ** -39 * size * a.sm_scale)
    bound = dz + 2.0 ** -22 * np.abs(want["lse"])
    assert (np.abs(lse - want["lse"]) <= bound).all(), (np.abs(lse - want["lse"]) / bound).max()
    # exp(2 dz) - 1 is the most that a weight changes by
    tol = 2.0 ** -8 * np.abs(want["out"]) + want["spread"] * (
        2.0 ** -11 + np.expm1(np.minimum(2 * dz, 30))[..., None]) * 1.01 + K * 2.0 ** -24
    assert (np.abs(out - want["out"]) <= tol).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,G,D,code", [(2, 4, 128, "int8"), (1, 16, 128, "int8"), (2, 1, 256, "e4m3"),
                                            (3, 9, 64, "e4m3"), (1, 6, 192, "int8")])
def test_attend_largest_weight_stays_whole(heads, G, D, code, dtype):
    """One live entry, of any scale: its V row comes out with the output's own rounding alone
    (and some 32-bit ones: exp2, log2, reciprocals)."""
    rng = np.random.default_rng(400 + D)
    for K in (1, 40):
        a = Attend(rng, 3, 2, K, heads, G, D, 8, code, dtype, holes=0)
        a.scales[:, :, 1] = rng.random(a.scales[:, :, 1].shape) + 0.1
        a.locs[:, :, 1:] = -1
        a.rows[a.locs[:, :, 0], :2 * heads * D] = random_codes(rng, (3, 2, 2 * heads * D), code)
        want = a.reference()["out"]
        got = a.run()[0].cpu().double().numpy()
        u = torch.finfo(a.q.dtype).eps / 2
        tol = (u + 2.0 ** -20) * np.abs(want) + (2.0 ** -25 if dtype == "fp16" else 0)
        assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / np.maximum(tol, 1e-30)).max()
