"""Calls around a decode step at the edges of what they accept."""
import numpy as np
import pytest
import torch

import kv_reference as kvref
import sparse_attention_kv_swap_gb300 as pkg
import step_reference as ref
from sparse_attention_kv_swap_gb300 import binding as B
from test_gpu_step import CODES, DTYPES, Prefix, Rotate, Select, dev, i32, randn

pytestmark = pytest.mark.gpu


# ---- shared prefixes, joined in place ---------------------------------------------------------

@pytest.mark.parametrize("B_,S,H,G,D,lens", [
    (64, 4, 8, 8, 128, [4096]),    # 1024 CTAs put rows together, 2 for each row: several waves
    (64, 4, 8, 8, 192, [2048]),    # 3
    (64, 4, 8, 8, 256, [2048]),    # 4
    (40, 4, 8, 8, 96, [3000, 1]),  # rows of one part beside rows of many
    (200, 2, 4, 4, 64, [900, 70, 0]),
    (4, 1, 2, 4, 256, [6000]),     # 16 for each row
    (2, 1, 1, 1, 128, [6000]),
])
def test_prefix_joined_in_place(B_, S, H, G, D, lens):
    """The same bits whether the outputs are the given ones, both or one of them, or lie apart; the
    CTAs that put a row together are not ordered.  Nothing past the workspace is written."""
    rng = np.random.default_rng(D + B_)
    a = Prefix(rng, B_, S, H, G, D, lens, 16, join=True)
    rows, scales = dev(a.rows), dev(a.scales)
    size = a.workspace().numel()
    ws = torch.full((size + 4096,), 255, dtype=torch.uint8, device="cuda")
    want = a.run(rows=rows, workspace=ws[:size])
    for out_too, lse_too in ((True, True), (False, True), (True, False)):
        for _ in range(3):
            join = (dev(a.join[0]), dev(a.join[1]))
            got = a.run(rows=rows, join=join, out=join[0] if out_too else None,
                        lse=join[1] if lse_too else None, workspace=ws[:size])
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (ws[size:] == 255).all()
    if B_ * S * H * G * lens[0] < 1 << 17:
        a.check(want)


def test_prefix_joined_in_place_without_prefixes():
    """Rows of no prefix keep what they are given, and an empty set is still zeros."""
    rng = np.random.default_rng(30)
    a = Prefix(rng, 300, 4, 8, 8, 128, [40], starts=[100, 101], join=True)
    want = a.run()
    out, lse = dev(a.join[0]), dev(a.join[1])
    got = a.run(join=(out, lse), out=out, lse=lse)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    none = torch.from_numpy(np.isneginf(a.join[1]))[101:]
    assert torch.equal(got[1].cpu()[101:], torch.from_numpy(a.join[1])[101:])
    assert (got[0].cpu()[101:][none] == 0).all()
    assert torch.equal(got[0].cpu()[101:][~none], a.join[0][101:][~none])


# ---- V scales that are far apart --------------------------------------------------------------

def prefix_with_scales(rng, B_, D, n, T, steps):
    """A call whose blocks' V scales have the logarithms `steps` (None: 0), over and over; equal
    logits, then ones that fall where V's scale rises."""
    a = Prefix(rng, B_, 1, 1, 4, D, [n], T)
    a.rows[0, :, :D] = 0x38  # 1.0 in every channel of K
    a.q = torch.zeros_like(a.q)
    a.q[..., 0] = 1.0
    at = [steps[i % len(steps)] for i in range(a.scales.shape[1])]
    log = np.array([x or 0.0 for x in at])
    a.scales[0, :, 1, 0] = np.where([x is not None for x in at], np.exp2(log), 0.0)
    for tilt in (0.0, -1.0):
        z = 8 + tilt * (log - log.min()) * np.log(2) / 40
        a.scales[0, :, 0, 0] = z * D ** 0.5
        yield a


@pytest.mark.parametrize("D,B_", [(64, 2), (128, 50), (192, 2)])
@pytest.mark.parametrize("steps", [40 * (-50,) + 300 * (87,), 300 * (-100,) + 40 * (100,),
                                   200 * (None,) + 200 * (50,) + 200 * (100,)])
def test_prefix_reference_jumps(D, B_, steps):
    """A token's weight in the sum stays when a later V scale, 2^137 and more times its own, moves the
    reference.  Blocks of 7 tokens, several tiles a CTA; the bounds are those of Prefix.check."""
    rng = np.random.default_rng(D)
    for a in prefix_with_scales(rng, B_, D, 7 * 9000, 7, steps):
        a.check(a.run())


# log2 of the V scales of consecutive blocks, repeated along the prefix.
STEPS = [(80, -59), (-59, 80), (-50, 87), (87, -50), (100, -100), (-100, 100), (49, -60),
         (51, -60), (-60, -61), (-61, 100, -60, 49), (100,) + 30 * (-59,), 30 * (-59,) + (100,),
         (None, 90, -90), (0, None, -59, 51)]


@pytest.mark.parametrize("T,n", [(16, 597), (16, 20005), (64, 40011)])
@pytest.mark.parametrize("D,B_", [(64, 2), (128, 34), (192, 2)])
def test_prefix_v_scales_in_steps(T, n, D, B_):
    """Blocks of 16 tokens and more, whose scales leave the softmax's loops: a token of a small V scale
    has its full weight whatever came before it, beside it in its tile or after it.  One tile a
    CTA, or several; the bounds are those of Prefix.check."""
    rng = np.random.default_rng(T + D)
    for steps in STEPS:
        for a in prefix_with_scales(rng, B_, D, n, T, steps):
            a.check(a.run())


# ---- the longest sequences ---------------------------------------------------------------------

def test_bounds_of_the_longest_sequence():
    """2^31 - 1 tokens, each of 32 elements that begin one element after the token before's."""
    M, T, D = 2 ** 31 - 1, 4096, 32
    gen = torch.Generator(device="cuda")
    gen.manual_seed(40)
    flat = torch.empty(M + D - 1, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    k = flat.as_strided((1, M, 1, D), (0, 1, 0, 1))
    got = torch.zeros(pkg.bounds_shape(1, M, T, 1, D), dtype=torch.bfloat16, device="cuda")
    pkg.hs_bound_keys(k, i32([0]), i32([0]), i32([M]), T, M, got)
    whole = M // T
    for d in range(D):
        x = flat[d:d + whole * T].view(whole, T)
        assert torch.equal(got[0, :whole, 0, 0, d], x.amin(1))
        assert torch.equal(got[0, :whole, 0, 1, d], x.amax(1))
        x = flat[d + whole * T:d + M]
        assert got[0, whole, 0, 0, d] == x.min() and got[0, whole, 0, 1, d] == x.max()
    # the last tokens alone, into the blocks as they are
    again = got.clone()
    n = 5000
    pkg.hs_bound_keys(k[:, M - n:], i32([0]), i32([M - n]), i32([n]), T, M, again)
    assert torch.equal(again, got)
    del flat, k, got, again, x
    torch.cuda.empty_cache()


def test_prefix_of_the_longest_store():
    """2^31 - 1 tokens of one head of 32, three tiles of rows: even rows give all their weight to the
    last thousand tokens, odd ones none.  A row's sums over a CTA's tokens are up to 441506 tiles of 2
    additions a thread, 2^-24 each, and of 4 products, 2^-23 each."""
    L, T, D, n, last = 2 ** 31 - 1, 4096, 32, 520, 1000
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("the store is 137 GB")
    fmt = pkg.make_kv_format(1, D, T)
    rows = torch.zeros((1, L, 2 * D), dtype=torch.uint8, device="cuda")
    rows[0, :, D:] = 0x38  # V: 1.0
    rows[0, -last:, 0] = 0x38  # K
    gen = torch.Generator(device="cuda")
    gen.manual_seed(41)
    v = torch.randn((last, D), device="cuda", generator=gen).to(torch.float8_e4m3fn)
    rows[0, -last:, D:] = v.view(torch.uint8)
    scales = torch.ones(fmt.scales_shape(1, L), device="cuda")
    q = torch.zeros((n, 1, 1, D), dtype=torch.float16, device="cuda")
    q[0::2, ..., 0], q[1::2, ..., 0] = 40.0, -40.0
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    ws = torch.empty(pkg.hs_prefix_workspace_bytes(fmt, n, 1, 1, 1), dtype=torch.uint8, device="cuda")
    pkg.hs_attend_prefix(fmt, q, rows, scales, i32([0]), i32([L]), i32([0, n]), out, lse=lse,
                         sm_scale=1.0, workspace=ws)
    torch.cuda.synchronize()
    # e^40 a token: the others' 2^31 together are under 2^-36 of it
    assert (lse[0::2] - (40 + np.log(last))).abs().max() < 1e-4
    assert (out[0::2].float() - v.float().mean(0)).abs().max() < 2e-3
    tol = 441506 * 2.0 ** -23
    assert (lse[1::2] - np.log(L - last)).abs().max() < tol + 1e-5
    assert (out[1::2].float() - 1).abs().max() < 5 * tol
    del rows, scales, q, out, lse, ws, v
    torch.cuda.empty_cache()


# ---- eviction and selection ----------------------------------------------------------------------

@pytest.mark.parametrize("code,dtype,T,each", [("e4m3", "bf16", 16, 16), ("int8", "fp16", 16, 8),
                                               ("int8", "bf16", 24, 32), ("e4m3", "fp16", 16, 7)])
def test_evict_makes_bounds_anew(code, dtype, T, each):
    """Of what is kept, as the host pool holds it; other requests' stay, and tokens that are appended
    later widen them.  Selection by them is that of the reference."""
    from sparse_attention_kv_swap_gb300.cache import SwapInCache
    rng = np.random.default_rng(each)
    R, L, heads, D, layers, blocks = 3, 120, 2, 64, 2, 3
    fmt = pkg.make_kv_format(heads, D, T, CODES[code])
    cache = SwapInCache(pkg.make_config(R, L, fmt.item_size_bytes, 8 * each, blocks * each, 1,
                                        num_layers=layers, extra_page_size=16))
    req, none = i32([0, 1, 2]), i32([0, 0, 0])
    lens = np.array([120, 75, 40])
    scales = [cache.kv_scales(fmt) for _ in range(layers)]
    bounds = [cache.key_bounds(fmt, DTYPES[dtype], each) for _ in range(layers)]
    acc = [dev(rng.random((R, L)).astype(np.float32)) for _ in range(layers)]
    for l in range(layers):
        k = dev(randn(rng, (R, L, heads, D), dtype))
        k[0, 5, 0, 3] = 60000.0  # fp16: the code's value is beyond the type
        cache.append_kv(fmt, scales[l], k, k, req, none, i32(lens), layer_id=l)
        cache.bound_keys(bounds[l], each, k, req, none, i32(lens))
        acc[l][0, 5] = 2.0  # kept
    want = [b.cpu() for b in bounds]
    budget = 50
    assert cache.evict(fmt, scales, acc, [0, 1], [120, 75], budget, 10, bounds=bounds,
                       block_tokens=each) == [50, 50]
    torch.cuda.synchronize()
    most = torch.finfo(DTYPES[dtype]).max
    for l in range(layers):
        x = torch.from_numpy(kvref.unpack(cache.host_pools[l][:2, :budget].numpy(), heads, D,
                                          code)[:, :, 0]).float()
        s = scales[l].cpu()[:2, np.arange(budget) // T, 0, :, None]
        keys = (x * s).clamp(-most, most).to(DTYPES[dtype])
        full = want[l].double().numpy()
        ref.bound(keys.double().numpy(), [0, 1], [0, 0], [budget, budget], each, L, full)
        assert np.array_equal(bounds[l].cpu().double().numpy(), full)
        # the next token, and a selection
        k = dev(randn(rng, (R, 1, heads, D), dtype))
        at = i32([50, 50, 40])
        cache.append_kv(fmt, scales[l], k, k, req, at, i32([1, 1, 1]), layer_id=l)
        cache.bound_keys(bounds[l], each, k, req, at, i32([1, 1, 1]))
        ref.bound(k.cpu().double().numpy(), [0, 1, 2], [50, 50, 40], [1, 1, 1], each, L, full)
        assert np.array_equal(bounds[l].cpu().double().numpy(), full)
        q = randn(rng, (R, 1, 4, D), dtype)
        got = cache.select_blocks(bounds[l], each, dev(q), req, i32([51, 51, 41]))["topk"]
        score, _ = ref.scores(q.double().numpy(), full, [0, 1, 2], [51, 51, 41], each, L)
        topk = ref.select(score, [51, 51, 41], [0, 1, 2], R, each, L, blocks, 1, 1)[1]
        assert np.array_equal(got.cpu().numpy(), topk)
    assert cache.status() == (B.HS_OK, 0)
    cache.close()


# ---- selection ---------------------------------------------------------------------------------

@pytest.mark.parametrize("up", [-40, 55])
def test_select_near_ties_of_small_and_large_scores(up):
    """Queries and bounds of 2^-40 and of 2^55: scores that differ by less than the sums in 32 bits can
    tell are told apart at the ends of the range too."""
    rng = np.random.default_rng(50)
    T, L = 4, 2400
    s = Select(rng, 2, 2, 4, 4, 64, T, L, 100, 1, 1)
    s.lens[:] = L
    s.bounds[:] = s.bounds[:1, :1]
    steps = torch.from_numpy(rng.integers(0, 128, (s.R, 600)) * 2.0 ** -7 + 1.0)
    s.bounds[:, :, 2, 0, 5] = 0
    s.bounds[:, :, 2, 1, 5] = (steps * 2.0 ** -14).to(torch.bfloat16)
    s.q[:, :, 8:12, 5] = 1.0
    plain = s.run()
    s.check(plain)
    s.q, s.bounds = s.q * 2.0 ** up, s.bounds * 2.0 ** up
    got = s.run()
    s.check(got)
    assert torch.equal(got[0], plain[0]) and torch.equal(got[2], plain[2] * 2.0 ** (2 * up))


# ---- norms and rotation ------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rotate_largest_elements(dtype):
    """Elements just under 2^59, the largest whose squares are promised to add up, beside small ones."""
    rng = np.random.default_rng(51)
    r = Rotate(rng, 1, 3, 4, 2, 256, 256, dtype)
    r.q = torch.full(r.q.shape, 255 * 2.0 ** 51, dtype=r.q.dtype)
    r.q[:, 1] = -r.q[:, 1]
    r.q[:, 2] *= 2.0 ** -100
    r.check(r.run())
