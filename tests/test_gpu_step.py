"""The calls around a decode step on the GPU against the plain implementation
(step_reference.py), within bounds that count their roundings; selections exactly."""
import numpy as np
import pytest
import torch

import sparse_attention_kv_swap_gb300 as pkg
import step_reference as ref
from sparse_attention_kv_swap_gb300 import binding as B

pytestmark = pytest.mark.gpu

CODES = {"e4m3": B.HS_KV_E4M3, "int8": B.HS_KV_INT8}
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def dev(x):
    return (torch.from_numpy(np.ascontiguousarray(x)) if isinstance(x, np.ndarray) else x).cuda()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def randn(rng, shape, dtype, size=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * size).to(DTYPES[dtype])


# ---- norms and rotation --------------------------------------------------------------

class Rotate:
    def __init__(self, rng, B_, M, Hq, Hkv, D, rot, dtype, adjacent=False, axes=1, norm=True,
                 far=40000):
        self.q, self.k = randn(rng, (B_, M, Hq, D), dtype), randn(rng, (B_, M, Hkv, D), dtype)
        self.freq = ref.frequencies(rot) if rot else []
        self.axis = [j % axes for j in range(rot // 2)]
        self.adjacent, self.dtype, self.D = adjacent, dtype, D
        self.pos = rng.integers(0, far, (axes, B_, M)).astype(np.int32)
        self.w = [1 + 0.3 * rng.standard_normal(D).astype(np.float32) if norm else None
                  for _ in range(2)]
        self.eps = 1e-5

    def rope(self):
        return pkg.make_rope(self.freq, self.axis, adjacent=self.adjacent) if self.freq else None

    def run(self, q=None, k=None, q_out=None, k_out=None, **kw):
        q, k = dev(self.q) if q is None else q, dev(self.k) if k is None else k
        q_out = torch.full_like(q, float("nan")) if q_out is None else q_out
        k_out = torch.full_like(k, float("nan")) if k_out is None else k_out
        w = [None if x is None else dev(x) for x in self.w]
        pkg.hs_norm_rope(q, k, dev(self.pos), self.rope(), q_out, k_out, q_weight=w[0],
                         k_weight=w[1], eps=self.eps, **kw)
        torch.cuda.synchronize()
        return q_out, k_out

    def check(self, got):
        """u is half a step of the output type.  In 32 bits: the mean of squares is off by 21 roundings
        of 2^-24 (half of that in its root), rsqrt by 2^-22 and the products by 3 of 2^-24,
        together under 2^-20; sine and cosine by 2^-22 (two units and the angle's 2^-25), two
        products and a sum of 2^-24 each: under 2^-20 of the pair's length too."""
        u = torch.finfo(DTYPES[self.dtype]).eps / 2
        for x, w, y in ((self.q, self.w[0], got[0]), (self.k, self.w[1], got[1])):
            want, size = ref.norm_rope(x.double().numpy(), w, self.eps, self.pos, self.freq,
                                       self.axis, self.adjacent)
            tol = u * np.abs(want) + size * 2.0 ** -19 * (1 + u) + (
                2.0 ** -25 if self.dtype == "fp16" else 1e-38)
            err = np.abs(y.cpu().double().numpy() - want)
            assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D", [32, 64, 96, 128, 192, 256])
@pytest.mark.parametrize("adjacent", [False, True])
def test_rotate_head_sizes(dtype, D, adjacent):
    rng = np.random.default_rng(D)
    for rot in {D, 16, D // 2 // 16 * 16, 0}:
        r = Rotate(rng, 2, 5, 6, 2, D, rot, dtype, adjacent)
        r.check(r.run())


@pytest.mark.parametrize("B_,M,Hq,Hkv", [(1, 1, 1, 1), (1, 1, 128, 1), (64, 1, 64, 8), (3, 1000, 1, 1),
                                         (1, 333, 15, 5), (200, 1, 5, 5), (2, 4000, 4, 2)])
def test_rotate_sizes(B_, M, Hq, Hkv):
    rng = np.random.default_rng(M)
    r = Rotate(rng, B_, M, Hq, Hkv, 64, 64, "bf16")
    r.check(r.run())


@pytest.mark.parametrize("axes", [2, 3, 4])
def test_rotate_axes(axes):
    rng = np.random.default_rng(axes)
    r = Rotate(rng, 3, 40, 4, 2, 128, 96, "fp32", axes=axes, adjacent=axes == 3)
    r.check(r.run())


@pytest.mark.parametrize("B_,M,Hq,Hkv,D,dtype", [(3, 5001, 3, 1, 64, "fp16"), (1, 12000, 1, 1, 32, "fp32"),
                                                 (700, 3, 2, 2, 128, "bf16"), (2, 37, 128, 120, 96, "bf16"),
                                                 (5000, 1, 2, 1, 192, "fp16"), (2, 911, 7, 5, 256, "fp32")])
def test_rotate_tiles(B_, M, Hq, Hkv, D, dtype):
    """Tiles and runs that do not divide the tokens, in one wave of CTAs and in several."""
    rng = np.random.default_rng(M)
    a = Rotate(rng, B_, M, Hq, Hkv, D, D // 2, dtype)
    count = rng.integers(0, M + 1, B_)
    count[0], count[1:2] = M, 0
    got = a.run(count=i32(count))
    want = a.run()
    a.check(want)
    on = torch.arange(M, device="cuda") < i32(count)[:, None]
    for x, y in zip(got, want):
        assert torch.equal(x[on], y[on]) and torch.isnan(x[~on]).all()


def test_rotate_without_norm_and_one_side():
    rng = np.random.default_rng(1)
    r = Rotate(rng, 2, 9, 4, 2, 64, 32, "fp16", norm=False)
    r.check(r.run())
    r.w[1] = np.ones(64, np.float32)  # keys alone are normalised
    both = r.run()
    r.check(both)
    q, k = dev(r.q), dev(r.k)
    out = torch.empty_like(q)
    pkg.hs_norm_rope(q, None, dev(r.pos)[0], r.rope(), out, None)
    assert torch.equal(out, both[0])
    out = torch.empty_like(k)
    pkg.hs_norm_rope(None, k, dev(r.pos), r.rope(), None, out, k_weight=dev(r.w[1]), eps=r.eps)
    assert torch.equal(out, both[1])


def test_rotate_far_and_negative_positions():
    """Angles of whole 64ths of a turn are known at every position: 32-bit ones included."""
    rng = np.random.default_rng(2)
    r = Rotate(rng, 1, 64, 2, 1, 64, 64, "fp32", norm=False)
    part = rng.integers(1, 64, 32)
    r.freq = [2 * np.pi * int(p) / 64 for p in part]
    far = rng.integers(-2 ** 31, 2 ** 31, (1, 1, 64))
    far[0, 0, :4] = [2 ** 31 - 1, -2 ** 31, -1, 0]
    r.pos = far.astype(np.int32)
    got = r.run()
    # the frequency is a double: off by 2^-53 of itself, 2^31 times that at the last position
    x = r.q.double().numpy()
    for j in range(32):
        angle = 2 * np.pi * ((far * int(part[j])) % 64)[0] / 64
        c, s = np.cos(angle)[..., None], np.sin(angle)[..., None]
        y0, y1 = got[0].cpu().double().numpy()[..., j], got[0].cpu().double().numpy()[..., j + 32]
        size = np.hypot(x[..., j], x[..., j + 32])
        tol = size * (2.0 ** -19 + 2.0 ** 31 * 2.0 ** -52 * r.freq[j])
        assert (np.abs(y0 - (x[..., j] * c - x[..., j + 32] * s)) <= tol).all()
        assert (np.abs(y1 - (x[..., j] * s + x[..., j + 32] * c)) <= tol).all()


def test_rotate_strides_in_place_and_counts():
    rng = np.random.default_rng(3)
    r = Rotate(rng, 3, 7, 4, 2, 64, 48, "bf16")
    plain = r.run()
    fused = torch.zeros((3, 7, 8, 80), dtype=torch.bfloat16, device="cuda")
    for off in (0, 1, 8):
        q, k = fused[:, :, :4, off:off + 64], fused[:, :, 4:6, off:off + 64]
        q.copy_(r.q)
        k.copy_(r.k)
        got = r.run(q=q, k=k)
        assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])
        before = fused.clone()
        r.run(q=q, k=k, q_out=q, k_out=k)  # in place
        assert torch.equal(q, plain[0]) and torch.equal(k, plain[1])
        q.copy_(r.q)
        k.copy_(r.k)
        assert torch.equal(fused, before)  # nothing else written
    turned = torch.zeros((4, 7, 3, 64), dtype=torch.bfloat16, device="cuda").permute(2, 1, 0, 3)
    r.run(q_out=turned)
    assert torch.equal(turned, plain[0])
    one = dev(r.k)[:, :, :1].expand(3, 7, 2, 64)  # one key for all heads (stride 0)
    r2 = Rotate(rng, 3, 7, 4, 2, 64, 48, "bf16")
    r2.q, r2.k, r2.pos, r2.w = r.q, one.cpu().contiguous(), r.pos, r.w
    r2.check(r2.run(k=one, k_out=torch.empty((3, 7, 2, 64), dtype=torch.bfloat16, device="cuda")))
    q_out = torch.full((3, 7, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    k_out = torch.full((3, 7, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    r.run(q_out=q_out, k_out=k_out, count=i32([0, 7, 3]))
    for b, n in ((0, 0), (1, 7), (2, 3)):
        assert torch.equal(q_out[b, :n], plain[0][b, :n]) and (q_out[b, n:] == 7).all()
        assert torch.equal(k_out[b, :n], plain[1][b, :n]) and (k_out[b, n:] == 7).all()
    r.run(count=i32([-5, 100, 2 ** 31 - 1]))


def test_rotate_special_values():
    """Zeros stay zero, an infinity or NaN spoils its own head only, large values do not overflow."""
    rng = np.random.default_rng(4)
    r = Rotate(rng, 1, 2, 4, 1, 64, 64, "fp32")
    clean = r.run()
    r.q[0, 0, 0] = 0
    r.q[0, 1, 2, 5] = float("nan")
    r.q[0, 1, 3, 5] = float("inf")
    got = r.run()
    assert (got[0][0, 0, 0] == 0).all() and torch.isnan(got[0][0, 1, 2]).all()
    assert torch.isnan(got[0][0, 1, 3]).any()
    assert torch.equal(got[0][0, 0, 1:], clean[0][0, 0, 1:])
    assert torch.equal(got[0][0, 1, :2], clean[0][0, 1, :2])
    r = Rotate(rng, 1, 2, 4, 1, 64, 64, "bf16")
    r.q = (r.q.double() * 1e15).to(torch.bfloat16)
    r.check(r.run())


# ---- bounds ----------------------------------------------------------------------------

def random_bounds(rng, R, NB, H, D, dtype):
    mid, wide = rng.standard_normal((2, R, NB, H, D))
    x = np.stack((mid - np.abs(wide), mid + np.abs(wide)), axis=3)
    return torch.from_numpy(x).to(DTYPES[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("H,D,T", [(1, 32, 1), (2, 64, 16), (5, 96, 7), (8, 128, 64), (3, 192, 48),
                                   (4, 256, 33), (1, 64, 4096), (32, 128, 16)])
@pytest.mark.parametrize("M", [1, 40, 300])
def test_bounds(dtype, H, D, T, M):
    rng = np.random.default_rng(H * D + M)
    R, L, n = 5, M + 210, 4
    k = randn(rng, (n, M, H, D), dtype)
    bounds = random_bounds(rng, R, -(-L // T), H, D, dtype)
    req = rng.permutation(R)[:n]
    start = np.array([0, T % 200, rng.integers(0, 200), L - M])
    count = np.array([M, M, rng.integers(0, M + 1), M])
    want = bounds.double().numpy()
    ref.bound(k.double().numpy(), req, start, count, T, L, want)
    got = dev(bounds)
    pkg.hs_bound_keys(dev(k), i32(req), i32(start), i32(count), T, L, got)
    assert np.array_equal(got.cpu().double().numpy(), want)


def test_bounds_token_by_token_and_in_one():
    rng = np.random.default_rng(5)
    R, L, H, D, T = 2, 100, 2, 64, 24
    k = randn(rng, (R, L, H, D), "bf16")
    one = torch.zeros((R, 5, H, 2, D), dtype=torch.bfloat16, device="cuda")
    each = torch.full_like(one, 9.0)
    pkg.hs_bound_keys(dev(k), i32([0, 1]), i32([0, 0]), i32([L, L]), T, L, one)
    for t in range(L):
        pkg.hs_bound_keys(dev(k)[:, t:t + 1], i32([0, 1]), i32([t, t]), i32([1, 1]), T, L, each)
    assert torch.equal(one, each)
    assert (one[:, :, :, 0] <= one[:, :, :, 1]).all()


def test_bounds_leaves_bad_entries_alone():
    rng = np.random.default_rng(6)
    R, L, H, D, T, M = 6, 64, 1, 64, 16, 8
    k = dev(randn(rng, (8, M, H, D), "fp16"))
    start = dev(random_bounds(rng, R, 4, H, D, "fp16"))
    got = start.clone()
    big = 2 ** 31 - 1
    pkg.hs_bound_keys(k, i32([-1, R, 0, 1, 2, 3, 4, 5]), i32([0, 0, -1, L - 3, big, 0, 0, 5]),
                      i32([8, 8, 8, 8, 8, M + 1, -1, 0]), T, L, got)
    assert torch.equal(got, start)


def test_bounds_nan_and_strides():
    rng = np.random.default_rng(7)
    L, H, D, T, M = 40, 3, 96, 16, 37
    wide = torch.zeros((2, M, H + 1, D + 16), dtype=torch.bfloat16, device="cuda")
    k = randn(rng, (2, M, H, D), "bf16")
    k[0, 3, 1, 5] = float("nan")
    k[1, :, 2, 7] = float("nan")
    k[1, 9, 0, 0] = float("inf")
    want = np.zeros((2, 3, H, 2, D))
    ref.bound(k.double().numpy(), [1, 0], [0, 3], [M, M], T, L, want)
    for off in (0, 1, 8):
        view = wide[:, :, 1:, off:off + D]
        view.copy_(k)
        got = torch.zeros((2, 3, H, 2, D), dtype=torch.bfloat16, device="cuda")
        pkg.hs_bound_keys(view, i32([1, 0]), i32([0, 3]), i32([M, M]), T, L, got)
        assert np.array_equal(got.cpu().double().numpy(), want)
    flat = torch.zeros(got.numel() + 1, dtype=torch.bfloat16, device="cuda")
    odd = flat[1:].view(got.shape)  # bounds off 16 bytes
    pkg.hs_bound_keys(view, i32([1, 0]), i32([0, 3]), i32([M, M]), T, L, odd)
    assert torch.equal(odd, got)


# ---- selection ---------------------------------------------------------------------------

class Select:
    def __init__(self, rng, B_, S, H, G, D, T, L, n, first=1, last=1, dtype="bf16", R=None):
        self.T, self.L, self.n, self.first, self.last = T, L, n, first, last
        self.R = R or B_ + 1
        self.q = randn(rng, (B_, S, H * G, D), dtype)
        self.bounds = random_bounds(rng, self.R, -(-L // T), H, D, dtype)
        self.req = rng.permutation(self.R)[:B_]
        self.lens = rng.integers(max(1, L // 2), L + 1, B_)
        self.lens[0] = L

    def run(self, q=None, bounds=None, stream=None, blocks=True):
        q = dev(self.q) if q is None else q
        bounds = dev(self.bounds) if bounds is None else bounds
        B_, S = q.shape[:2]
        topk = torch.full((B_, S, self.n * self.T), -7, dtype=torch.int32, device="cuda")
        out = torch.full((B_, S, self.n), -7, dtype=torch.int32, device="cuda") if blocks else None
        scores = torch.full((B_, S, bounds.shape[1]), float("nan"), device="cuda")
        ws = torch.full((max(1, pkg.hs_select_workspace_bytes(B_, S, self.L, self.T)),), 255,
                        dtype=torch.uint8, device="cuda")
        pkg.hs_select_blocks(q, bounds, i32(self.req), i32(self.lens), self.T, self.L, self.first,
                             self.last, out, topk, scores, ws, stream=stream)
        torch.cuda.synchronize()
        return out, topk, scores

    def check(self, got):
        """A score is a sum whose terms pass through one rounding of Q, the 8 products of a lane for
        each of its slices, 5 additions over lanes and 8 over warps, 2^-24 of the sum of magnitudes
        each."""
        q, bounds = self.q.double().numpy(), self.bounds.double().numpy()
        want, size = ref.scores(q, bounds, self.req, self.lens, self.T, self.L)
        blocks, topk = ref.select(want, self.lens, self.req, self.R, self.T, self.L, self.n,
                                  self.first, self.last)
        row = 2 * bounds.shape[2] * bounds.shape[4]
        z = got[2].cpu().double().numpy()
        assert np.array_equal(np.isneginf(z), np.isneginf(want))
        live = ~np.isneginf(want)
        err = np.abs(z[live] - want[live])
        assert (err <= (22 + row / 256) * 2.0 ** -24 * size[live]).all()
        if got[0] is not None:
            assert np.array_equal(got[0].cpu().numpy(), blocks)
        assert np.array_equal(got[1].cpu().numpy(), topk)


@pytest.mark.parametrize("S", [1, 2, 3, 4])
@pytest.mark.parametrize("H,G,D,T,L,n", [(1, 1, 32, 1, 40, 9), (2, 4, 64, 16, 4096, 32),
                                         (5, 3, 96, 48, 5000, 20), (8, 8, 128, 64, 3000, 17),
                                         (3, 6, 192, 32, 2000, 9), (1, 16, 256, 7, 1500, 50),
                                         (16, 2, 128, 128, 20000, 30), (1, 128, 64, 16, 900, 8)])
def test_select_sizes(S, H, G, D, T, L, n):
    rng = np.random.default_rng(S + D)
    s = Select(rng, 3, S, H, G, D, T, L, n, dtype="bf16" if S % 2 else "fp16")
    s.check(s.run())


@pytest.mark.parametrize("S,H,D,L,T", [(1, 64, 128, 700, 16), (2, 32, 256, 300, 8), (4, 16, 256, 260, 4),
                                       (1, 1, 64, 16384, 1), (4, 2, 64, 65536, 4)])
def test_select_largest(S, H, D, L, T):
    rng = np.random.default_rng(L)
    s = Select(rng, 1, S, H, 1, D, T, L, 64, 3, 5)
    s.check(s.run())


@pytest.mark.parametrize("S,H,D,L,T", [(1, 1, 32, 700, 4), (1, 64, 128, 9000, 8), (2, 16, 128, 20000, 128),
                                       (4, 16, 256, 2500, 16), (3, 20, 128, 70, 1), (2, 1, 64, 5, 16)])
def test_select_stays_in_workspace(S, H, D, L, T):
    rng = np.random.default_rng(L + S)
    B_ = 2
    s = Select(rng, B_, S, H, 1, D, T, L, 9)
    size = pkg.hs_select_workspace_bytes(B_, S, L, T)
    ws = torch.full((size + 4096,), 255, dtype=torch.uint8, device="cuda")
    topk = torch.full((B_, S, 9 * T), -7, dtype=torch.int32, device="cuda")
    out = torch.full((B_, S, 9), -7, dtype=torch.int32, device="cuda")
    scores = torch.full((B_, S, -(-L // T)), float("nan"), device="cuda")
    pkg.hs_select_blocks(dev(s.q), dev(s.bounds), i32(s.req), i32(s.lens), T, L, 1, 1, out, topk,
                         scores, ws[:size])
    s.check((out, topk, scores))
    assert (ws[size:] == 255).all()


@pytest.mark.parametrize("first,last,n", [(0, 0, 1), (0, 0, 12), (5, 0, 5), (0, 5, 5), (2, 3, 5),
                                          (1, 2, 30), (0, 1, 31), (0, 0, 32), (3, 3, 33), (1, 1, 100)])
def test_select_first_and_last(first, last, n):
    """Of up to 32 blocks; the last one is partly filled."""
    rng = np.random.default_rng(n)
    s = Select(rng, 6, 2, 2, 2, 64, 16, 510, n, first, last)
    s.lens = np.array([510, 509, 16 * n, 16 * n + 1, 1, 200])
    s.lens = np.clip(s.lens, 1, 600)  # 600: longer than the store
    s.check(s.run())


def test_select_empty_and_bad_requests():
    rng = np.random.default_rng(8)
    s = Select(rng, 6, 2, 2, 4, 64, 16, 400, 8)
    s.lens[1], s.lens[2] = 0, -3
    s.req[3], s.req[4] = -1, s.R
    got = s.run()
    s.check(got)
    for b in (1, 2, 3, 4):
        assert (got[0][b] == -1).all() and (got[1][b] == -1).all()
        assert torch.isneginf(got[2][b]).all()


@pytest.mark.parametrize("T", [1, 16])
def test_select_ties_and_near_ties(T):
    """Blocks of equal scores go by their order; scores that differ by less than the sums in 32 bits
    can tell are told apart."""
    rng = np.random.default_rng(9)
    L = 600 * T
    s = Select(rng, 3, 2, 4, 4, 64, T, L, 100, 1, 1)
    s.lens[:] = L
    s.bounds[:] = s.bounds[:1, :1]  # all blocks alike
    s.check(s.run())
    # one small channel differs by steps of 2^-8 of it, far below the sum's last place
    steps = torch.from_numpy(rng.integers(0, 128, (s.R, 600)) * 2.0 ** -7 + 1.0)
    s.bounds[:, :, 2, 0, 5] = 0
    s.bounds[:, :, 2, 1, 5] = (steps * 2.0 ** -14).to(torch.bfloat16)
    s.q[:, :, 8:12, 5] = 1.0
    z, _ = ref.scores(s.q.double().numpy(), s.bounds.double().numpy(), s.req, s.lens, T, L)
    gap = np.diff(np.sort(z[0, 0]))
    assert 0 < gap[gap > 0].min() < np.abs(z).max() * 2.0 ** -24
    s.check(s.run())


def test_select_special_values():
    """NaN scores come last; infinite bounds come first, and nothing hangs on them."""
    rng = np.random.default_rng(10)
    s = Select(rng, 1, 1, 1, 1, 64, 8, 800, 10, 0, 0)
    s.q = s.q.abs() + 0.5
    s.bounds[:, 3, 0, 1, 4] = float("nan")
    s.bounds[:, 7, 0, 1, 4] = float("inf")
    out, _, scores = s.run()
    assert torch.isnan(scores[0, 0, 3]) and torch.isposinf(scores[0, 0, 7])
    assert 7 in out.cpu() and 3 not in out.cpu()
    s.bounds[:, :, 0, 1, 4] = float("nan")
    out, _, _ = s.run()
    assert out.cpu().flatten().tolist() == list(range(10))


def test_select_strides_and_alignment():
    rng = np.random.default_rng(11)
    s = Select(rng, 3, 2, 2, 3, 96, 16, 700, 9)
    plain = s.run()
    s.check(plain)
    wide = torch.zeros((3, 2, 8, 112), dtype=torch.bfloat16, device="cuda")
    for off in (0, 1, 8):
        q = wide[:, :, 1:7, off:off + 96]
        q.copy_(s.q)
        for x, y in zip(s.run(q=q), plain):
            assert torch.equal(x, y)
    flat = torch.zeros(s.bounds.numel() + 1, dtype=torch.bfloat16, device="cuda")
    odd = flat[1:].view(s.bounds.shape)
    odd.copy_(s.bounds)
    for x, y in zip(s.run(bounds=odd), plain):
        assert torch.equal(x, y)
    assert torch.equal(s.run(blocks=False)[1], plain[1])


def test_select_reads_no_bounds_past_the_sequence():
    rng = np.random.default_rng(12)
    s = Select(rng, 2, 1, 2, 2, 64, 16, 640, 6)
    s.lens = np.array([100, 333])
    plain = s.run()
    for b in range(2):
        s.bounds[s.req[b], -(-s.lens[b] // 16):] = float("nan")
    for x, y in zip(s.run(), plain):
        assert torch.equal(x, y)


# ---- shared prefixes ------------------------------------------------------------------------

def random_codes(rng, shape, code):
    x = rng.standard_normal(shape).astype(np.float32)
    if code == "int8":
        return np.clip(np.rint(x * 40), -127, 127).astype(np.int8).view(np.uint8)
    t = torch.from_numpy(x * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
    return t.view(torch.uint8).numpy()


class Prefix:
    """Inputs of one hs_attend_prefix call; rows past the prefixes' lengths hold NaN codes."""

    def __init__(self, rng, B_, S, H, G, D, lens, T=16, code="e4m3", dtype="bf16", starts=None,
                 join=False, L=None, pad=0):
        self.H, self.G, self.D, self.T, self.code, self.dtype = H, G, D, T, code, dtype
        P = len(lens)
        self.lens = np.array(lens)
        self.L, self.R = L or max(1, self.lens.max(initial=1)), max(1, P)
        W = 2 * H * D + pad
        self.fmt = pkg.make_kv_format(H, D, T, CODES[code], W)
        self.q = randn(rng, (B_, S, H * G, D), dtype)
        self.prefix = rng.permutation(self.R)[:P]
        self.starts = np.arange(P + 1) * B_ // max(P, 1) if starts is None else np.array(starts)
        self.rows = random_codes(rng, (self.R, self.L, W), code)
        for p in range(P):
            if 0 <= self.lens[p] < self.L:
                self.rows[self.prefix[p], self.lens[p]:] = 0x7F
        shape = self.fmt.scales_shape(self.R, self.L)
        if code == "e4m3":
            self.scales = np.exp2(rng.integers(-9, -5, shape)).astype(np.float32)
        else:
            self.scales = (rng.random(shape) * 0.05 + 0.01).astype(np.float32)
        self.sm_scale = D ** -0.5
        self.join = None
        if join:
            lse = (np.log(self.L) + rng.standard_normal((B_, S, H * G))).astype(np.float32)
            lse[rng.random(lse.shape) < 0.2] = -np.inf
            out = randn(rng, (B_, S, H * G, D), dtype, 0.3)
            out[torch.from_numpy(np.isneginf(lse))] = float("nan")  # not to be read
            self.join = (out, lse)

    def reference(self):
        join = None
        if self.join is not None:
            join = (np.nan_to_num(self.join[0].double().numpy()), self.join[1].astype(np.float64))
        return ref.attend(self.q.double().numpy(), self.rows, self.scales, self.prefix, self.lens,
                          self.starts, self.T, self.H, self.code, self.sm_scale, join)

    def workspace(self):
        B_, S, Hq, _ = self.q.shape
        n = pkg.hs_prefix_workspace_bytes(self.fmt, B_, S, Hq, len(self.lens))
        return torch.full((n,), 255, dtype=torch.uint8, device="cuda")

    def run(self, q=None, out=None, join=None, rows=None, workspace=None, stream=None, lse=None):
        q = dev(self.q) if q is None else q
        out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda") if out is None else out
        lse = torch.full(q.shape[:3], float("nan"), device="cuda") if lse is None else lse
        if join is None and self.join is not None:
            join = (dev(self.join[0]), dev(self.join[1]))
        pkg.hs_attend_prefix(self.fmt, q, dev(self.rows) if rows is None else rows, dev(self.scales),
                             i32(self.prefix), i32(self.lens), i32(self.starts), out, lse=lse,
                             join_out=None if join is None else join[0],
                             join_lse=None if join is None else join[1], sm_scale=self.sm_scale,
                             workspace=self.workspace() if workspace is None else workspace,
                             stream=stream)
        torch.cuda.synchronize()
        return out, lse

    def check(self, got, want=None):
        """Bounds: u is half a step of the output type; a weight times its V scale carries f16's half
        step 2^-11 into the product, or 2^-36 of the largest one (2^-35 with the headroom
        of the reference); a logit is a sum of D exact products, each addition off by 2^-23 at most, times
        three 32-bit factors; exp2, the join's exp, log and division and the sums add under 2^-19
        and n * 2^-24."""
        want = want or self.reference()
        n = int(self.lens.max(initial=0))
        dz = (self.D + 8) * 2.0 ** -23 * want["logit"] + 2.0 ** -19 + n * 2.0 ** -24
        u = torch.finfo(DTYPES[self.dtype]).eps / 2
        tol = (u * np.abs(want["out"]) + want["spread"] * (2.0 ** -11 + 2 * dz[..., None]) * (1 + u)
               + n * (2.0 ** -24 + 2.0 ** -35) * want["biggest"]
               + (2.0 ** -24 if self.dtype == "fp16" else 1e-37))
        out, lse = (x.cpu().double().numpy() for x in got)
        err = np.abs(out - want["out"])
        assert (err <= tol).all(), (err / tol).max()
        empty = np.isneginf(want["lse"])
        assert (np.isneginf(lse) == empty).all()
        bad = np.abs(np.where(empty, 0, lse) - np.where(empty, 0, want["lse"]))
        bound = dz + 2.0 ** -22 * np.abs(np.where(empty, 0, want["lse"]))
        assert (bad <= bound).all(), (bad / bound).max()


@pytest.mark.parametrize("n", [1, 2, 15, 63, 64, 65, 127, 128, 129, 255, 257, 640, 5000])
@pytest.mark.parametrize("D,G", [(64, 4), (128, 150 // 2), (192, 3)])
def test_prefix_lengths(n, D, G):
    rng = np.random.default_rng(n + D)
    a = Prefix(rng, 2, 2, 1, G, D, [n])
    a.check(a.run())


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("D", [32, 64, 96, 128, 192, 256])
@pytest.mark.parametrize("H,G,dtype,B_", [(2, 4, "bf16", 3), (1, 16, "fp16", 17), (3, 5, "fp16", 30)])
def test_prefix_head_sizes(code, D, H, G, dtype, B_):
    rng = np.random.default_rng(D + G)
    a = Prefix(rng, B_, 1, H, G, D, [700], 24, code, dtype, join=D % 64 == 0)
    a.check(a.run())


@pytest.mark.parametrize("T", [1, 7, 24, 40, 64])
@pytest.mark.parametrize("B_,code", [(2, "e4m3"), (50, "int8")])
def test_prefix_block_sizes(T, B_, code):
    """Scales by 16 tokens and by token, rows of one tile and of two."""
    rng = np.random.default_rng(T)
    a = Prefix(rng, B_, 1, 2, 4, 64, [4000 - T], T=T, code=code)
    a.check(a.run())


@pytest.mark.parametrize("H,G", [(1, 1), (1, 128), (5, 3), (12, 4), (32, 1), (128, 1), (2, 17)])
def test_prefix_head_layouts(H, G):
    rng = np.random.default_rng(H * 200 + G)
    a = Prefix(rng, 2, 3, H, G, 64, [333], 7, "e4m3", "fp16", join=True)
    a.check(a.run())


@pytest.mark.parametrize("B_,S", [(1, 1), (1, 4), (33, 1), (16, 4), (17, 4), (64, 4), (130, 1)])
@pytest.mark.parametrize("G", [1, 8])
def test_prefix_batches(B_, S, G):
    """Row tiles of every fill: 1 to 2048 rows of a K/V head."""
    rng = np.random.default_rng(B_ * S + G)
    a = Prefix(rng, B_, S, 2, G, 64, [400], 32, "int8", "bf16")
    a.check(a.run())


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("join", [False, True])
def test_prefix_groups(D, join):
    """Prefixes of all lengths, of no tokens and of no requests; requests of no prefix; bad ones."""
    rng = np.random.default_rng(13)
    starts = [1, 4, 4, 9, 10, 10, 31, 31, 33, 34, 36]
    lens = [100, 50, 257, 1, 3, 0, 70, 900, -4, 5000]
    a = Prefix(rng, 40, 1, 2, 8, D, lens, starts=starts, join=join, L=900)
    a.prefix[7] = a.R  # rows 31 and 32
    got = a.run()
    a.check(got)
    if not join:
        for lo, hi in ((0, 1), (10, 31), (31, 34), (36, 40)):
            assert (got[0][lo:hi] == 0).all() and torch.isneginf(got[1][lo:hi]).all()
    a.starts = np.array([-5, 2, 30, 20, 25, 60, 10, 2 ** 31 - 1, -2 ** 31, 12, 40])  # not ascending
    a.check(a.run())


def test_prefix_most_groups():
    rng = np.random.default_rng(14)
    P = B.HS_MAX_PREFIXES
    a = Prefix(rng, 300, 1, 1, 2, 32, list(rng.integers(0, 300, P)), T=64)
    a.starts = np.sort(rng.integers(0, 301, P + 1))
    a.check(a.run())


def test_prefix_without_prefixes_is_the_join():
    rng = np.random.default_rng(15)
    a = Prefix(rng, 3, 2, 2, 2, 64, [], join=True)
    out, lse = a.run()
    none = torch.from_numpy(np.isneginf(a.join[1]))
    assert torch.equal(lse.cpu(), torch.from_numpy(a.join[1]))
    assert torch.equal(out.cpu()[~none], a.join[0][~none]) and (out.cpu()[none] == 0).all()
    a.join = None
    out, lse = a.run()
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_prefix_refuses_rows_in_host_memory():
    a = Prefix(np.random.default_rng(3), 2, 1, 1, 2, 64, [40])
    out = torch.full(a.q.shape, 7.0, dtype=a.q.dtype, device="cuda")
    for rows in (torch.from_numpy(a.rows), torch.from_numpy(a.rows).pin_memory()):
        with pytest.raises(ValueError):
            a.run(out=out, rows=rows)
    assert (out == 7).all()


def test_prefix_joined_in_place_and_strides():
    rng = np.random.default_rng(16)
    for lens, B_ in (([500], 3), ([90], 90), ([3000, 10], 5)):
        a = Prefix(rng, B_, 2, 2, 2, 64, lens, dtype="fp16", join=True)
        want = a.reference()
        plain = a.run()
        a.check(plain, want)
        out, lse = dev(a.join[0]), dev(a.join[1])
        got = a.run(out=out, lse=lse, join=(out, lse))
        assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])
        wide = torch.zeros((B_, 2, 6, 80), dtype=torch.float16, device="cuda")
        for off in (0, 1, 4, 8):
            q = wide[:, :, 1:5, off:off + 64]
            q.copy_(a.q)
            out = torch.zeros((4, 2, B_, 100), dtype=torch.float16, device="cuda").permute(2, 1, 0, 3)
            view = out[..., off:off + 64]
            view.copy_(a.join[0])
            got = a.run(q=q, out=view, join=(view, dev(a.join[1])))
            assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])
            assert (out[..., :off] == 0).all() and (out[..., off + 64:] == 0).all()
    assert torch.equal(a.run(lse=torch.empty_like(plain[1]))[0], plain[0])


def test_prefix_large_logits_and_scales():
    """Logits of hundreds, V scales that differ by 2^12, and scales of zero."""
    rng = np.random.default_rng(17)
    a = Prefix(rng, 3, 1, 1, 64, 128, [777], 8)
    a.q = a.q * 60
    a.scales[:, :, 1] = np.exp2(rng.integers(-12, 1, a.scales[:, :, 1].shape))
    a.scales[:, ::5, 1] = 0
    a.scales[:, ::7, 0] = 0
    a.check(a.run())
    a.sm_scale = -a.sm_scale
    a.check(a.run())
    a.sm_scale = 0.0
    a.check(a.run())


@pytest.mark.parametrize("D", [64, 192])
@pytest.mark.parametrize("order", [1, -1])
def test_prefix_v_scales_of_any_size(D, order):
    """The heaviest tokens have V scales far from the largest: the rounding follows the largest term.
    K and V scales per token; the logits rise or fall along the prefix, so that the reference moves."""
    rng = np.random.default_rng(18)
    a = Prefix(rng, 2, 1, 1, 4, D, [600], 1)
    ramp = np.linspace(0, 1, 600)[::order]
    for low, high in ((-100, -100), (-95, -60), (60, 100), (-30, 30), (-70, 10)):
        e = np.round(low + (high - low) * ramp)
        a.scales[0, :, 1, 0] = np.exp2(e)
        for tilt in (0.0, 2.0, -2.0):  # logits that rise as V falls, or with it
            a.rows[0, :, :D] = 0x38  # 1.0 in every channel of K
            a.scales[0, :, 0, 0] = 2.0 ** -6
            a.q = torch.zeros_like(a.q)
            a.q[..., 0] = 1.0
            z = tilt * (e - low) * np.log(2) / 2
            a.scales[0, :, 0, 0] = z * D ** 0.5
            a.check(a.run())
    a.scales[0, :, 1, 0] = 0  # nothing but zeros
    out, lse = got = a.run()
    a.check(got)
    assert (out == 0).all() and torch.isfinite(lse).all()


def test_prefix_query_magnitudes():
    """bf16 queries far outside f16's range, tiny ones and zeros."""
    rng = np.random.default_rng(19)
    a = Prefix(rng, 1, 1, 1, 4, 64, [300])
    q = a.q.double()
    q[0, 0, 0] *= 1e30
    q[0, 0, 1] *= 1e-30
    q[0, 0, 2] = 0
    a.q = q.to(torch.bfloat16)
    a.sm_scale = 1e-30
    a.check(a.run())
    a.sm_scale = 1.0
    a.q[0, 0, 0] = 0
    a.check(a.run())


@pytest.mark.parametrize("B_", [2, 80])
def test_prefix_nan_stays_in_its_head(B_):
    rng = np.random.default_rng(20)
    a = Prefix(rng, B_, 1, 2, 4, 64, [200])
    clean = a.run()
    a.q[0, 0, 1, 3] = float("nan")
    a.q[0, 0, 6, 3] = float("inf")
    out, lse = a.run()
    assert torch.isnan(out[0, 0, 1]).all() and torch.isnan(lse[0, 0, 1])
    assert torch.isnan(out[0, 0, 6]).any()
    for i in (0, 2, 3, 4, 5, 7):
        assert torch.equal(out[0, 0, i], clean[0][0, 0, i])
    assert torch.equal(out[1:], clean[0][1:])
    a.q[0, 0, 1, 3], a.q[0, 0, 6, 3] = 0, 0
    a.rows[0, 150, 64 + 5] = 0x7F  # K of head 1
    out, lse = a.run()
    assert torch.isnan(out[:, :, 4:]).all() and torch.isfinite(out[:, :, :4]).all()


def test_prefix_row_width_and_far_rows():
    """Padded rows, and rows whose byte offsets pass 32 bits."""
    rng = np.random.default_rng(21)
    a = Prefix(rng, 3, 1, 5, 4, 64, [333], pad=16)
    assert a.fmt.item_size_bytes == 656
    a.check(a.run())
    a = Prefix(rng, 2, 1, 8, 2, 128, [300], 64)
    want = a.run()
    big = torch.full((3, 1 << 20, 2048), 0x7F, dtype=torch.uint8, device="cuda")
    big[2, :300] = dev(a.rows)[0]
    scales = torch.full((3, (1 << 20) // 64, 2, 8), float("nan"), device="cuda")
    scales[2, :5] = dev(a.scales)[0]
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    pkg.hs_attend_prefix(a.fmt, dev(a.q), big, scales, i32([2]), i32([300]), i32([0, 2]), out, lse=lse,
                         workspace=a.workspace())
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_prefix_is_hs_attend_over_all_tokens():
    """The same attention as hs_attend's over a selection of all tokens, within both bounds."""
    rng = np.random.default_rng(22)
    a = Prefix(rng, 3, 1, 2, 4, 128, [500], dtype="fp16")
    out, lse = a.run()
    locs = torch.arange(500, dtype=torch.int32, device="cuda").expand(3, 1, 500).contiguous()
    got, got_lse = torch.empty_like(out), torch.empty_like(lse)
    pkg.hs_attend(a.fmt, dev(a.q), dev(a.rows)[0], locs, locs, i32([0, 0, 0]), dev(a.scales), a.L, got,
                  lse=got_lse)
    assert (got.float() - out.float()).abs().max() < 4e-3
    assert (got_lse - lse).abs().max() < 1e-4


# ---- streams, graphs, the whole step -------------------------------------------------------------

def calls(rng):
    """One call of every operator: (outputs to compare, function of a stream)."""
    r = Rotate(rng, 5, 3, 8, 2, 64, 64, "bf16")
    s = Select(rng, 5, 2, 2, 4, 64, 16, 3000, 20)
    p = Prefix(rng, 40, 1, 2, 4, 64, [900, 77], join=True)
    q, k, pos, rope = dev(r.q), dev(r.k), dev(r.pos), r.rope()
    w = [dev(x) for x in r.w]
    sq, bounds, sreq, slens = dev(s.q), dev(s.bounds), i32(s.req), i32(s.lens)
    key = dev(randn(rng, (5, 100, 2, 64), "bf16"))
    start, count = i32([0, 3, 50, 7, 100]), i32([100, 50, 1, 99, 100])
    pq, rows, scales = dev(p.q), dev(p.rows), dev(p.scales)
    prefix, lens, starts = i32(p.prefix), i32(p.lens), i32(p.starts)
    join = (dev(p.join[0]), dev(p.join[1]))

    def outputs():
        return [torch.zeros_like(q), torch.zeros_like(k), bounds.clone(),
                torch.zeros((5, 2, 20), dtype=torch.int32, device="cuda"),
                torch.zeros((5, 2, 320), dtype=torch.int32, device="cuda"),
                torch.zeros((5, 2, bounds.shape[1]), device="cuda"), torch.zeros_like(pq),
                torch.zeros(pq.shape[:3], device="cuda"),
                torch.zeros(pkg.hs_select_workspace_bytes(5, 2, 3000, 16), dtype=torch.uint8,
                            device="cuda"), p.workspace()]

    def call(o, stream=None):
        pkg.hs_norm_rope(q, k, pos, rope, o[0], o[1], w[0], w[1], stream=stream)
        pkg.hs_bound_keys(key, sreq, start, count, 16, 3000, o[2], stream=stream)
        pkg.hs_select_blocks(sq, o[2], sreq, slens, 16, 3000, 1, 1, o[3], o[4], o[5], o[8],
                             stream=stream)
        pkg.hs_attend_prefix(p.fmt, pq, rows, scales, prefix, lens, starts, o[6], lse=o[7],
                             join_out=join[0], join_lse=join[1], workspace=o[9], stream=stream)

    return outputs, call


def test_step_repeats_streams_and_graphs():
    """The same bits on every run, on another stream, replayed from a graph, and from two graphs and
    two streams at once with workspaces of their own."""
    outputs, call = calls(np.random.default_rng(23))
    first = outputs()
    call(first)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    again = outputs()
    side.wait_stream(torch.cuda.current_stream())
    call(again, stream=side)
    side.synchronize()
    held, graphs = [outputs(), outputs()], []
    for o in held:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(o)
        graphs.append(g)
    for _ in range(3):
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
    torch.cuda.synchronize()
    for other in [again] + held:
        for x, y in zip(first[:8], other[:8]):
            assert torch.equal(x, y)


@pytest.mark.parametrize("code,dtype,heads,group,D,T", [("e4m3", "bf16", 2, 4, 64, 16),
                                                        ("int8", "fp16", 3, 2, 96, 16)])
def test_decode_example(code, dtype, heads, group, D, T):
    """The example's loop, each call by the tensors it was given: rotated heads within their bounds,
    codes, scales, key bounds and selection exactly, the attention over the selected rows and the
    one joined with the shared prompt's within their bounds."""
    import importlib.util
    import pathlib
    import kv_reference as kvref
    path = pathlib.Path(__file__).resolve().parent.parent / "examples" / "decode_selected.py"
    spec = importlib.util.spec_from_file_location("decode_selected", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    rng = np.random.default_rng(25)
    R, limit, shared, blocks = 3, 150, 77, 4
    d = example.SelectingDecoder(R, limit, shared, blocks, heads, group, D, T, CODES[code],
                                 DTYPES[dtype])
    d.weight = [dev(1 + 0.3 * rng.standard_normal(D).astype(np.float32)) for _ in range(2)]
    pool = d.cache.host_pools[0]
    pool.zero_()
    rows, scales = pool.clone(), torch.zeros_like(d.scales, device="cpu")
    bounds = d.bounds.cpu().double().numpy()
    req = np.arange(R, dtype=np.int32)

    def turned(x, w, first, got):
        r = Rotate.__new__(Rotate)
        r.freq, r.axis, r.adjacent = ref.frequencies(D), [0] * (D // 2), False
        r.dtype, r.D, r.eps, r.w = dtype, D, 1e-6, [w, w]
        r.pos = (np.asarray(first)[:, None] + np.arange(x.shape[1])).astype(np.int32)[None]
        r.q = r.k = x
        r.check((got, got))

    def append(k, v, start, count):
        kvref.quantize(k, v, req, start, count, rows, scales, T, code)
        ref.bound(k.double().numpy(), req, start, count, T, limit, bounds)
        assert torch.equal(pool, rows) and torch.equal(d.scales.cpu(), scales)
        assert np.array_equal(d.bounds.cpu().double().numpy(), bounds)

    w = [x.cpu().numpy() for x in d.weight]
    k, v = randn(rng, (1, shared, heads, D), dtype), randn(rng, (1, shared, heads, D), dtype)
    ks = d.share(dev(k), dev(v))
    turned(k, w[1], [0], ks)
    srows, sscales = torch.zeros_like(d.rows, device="cpu"), torch.zeros_like(d.shared_scales,
                                                                             device="cpu")
    kvref.quantize(ks.cpu(), v, [0], [0], [shared], srows, sscales, T, code)
    assert torch.equal(d.rows.cpu(), srows) and torch.equal(d.shared_scales.cpu(), sscales)
    lens = np.array([140, 9, 97], dtype=np.int32)
    k, v = randn(rng, (R, 140, heads, D), dtype), randn(rng, (R, 140, heads, D), dtype)
    ks = d.prompt(dev(k), dev(v), i32(lens))
    torch.cuda.synchronize()
    turned(k, w[1], [shared] * R, ks)
    append(ks.cpu(), v, [0] * R, lens)
    for step in range(10):
        q = randn(rng, (R, 1, heads * group, D), dtype)
        k, v = randn(rng, (R, 1, heads, D), dtype), randn(rng, (R, 1, heads, D), dtype)
        d.step(dev(q), dev(k), dev(v))
        torch.cuda.synchronize()
        turned(q, w[0], shared + lens, d.q)
        turned(k, w[1], shared + lens, d.k)
        append(d.k.cpu(), v, lens, [1] * R)
        lens += 1
        dq = d.q.cpu().double().numpy()
        score, _ = ref.scores(dq, bounds, req, lens, T, limit)
        topk = ref.select(score, lens, req, R, T, limit, blocks, 1, 1)[1]
        assert np.array_equal(d.selected["topk"].cpu().numpy(), topk)
        # over the selected rows, as one prefix for each request
        a = Prefix.__new__(Prefix)
        a.H, a.G, a.D, a.T, a.code, a.dtype = heads, group, D, T, code, dtype
        a.lens = np.array([(topk[b] >= 0).sum() for b in range(R)])
        part = [ref.attend(dq[b:b + 1], rows[b:b + 1].numpy()[:, topk[b, 0, :a.lens[b]]],
                           np.ascontiguousarray(scales[b:b + 1].numpy()[:, topk[b, 0, :a.lens[b]] // T]),
                           [0], [a.lens[b]], [0, 1], 1, heads, code, D ** -0.5) for b in range(R)]
        want = {x: np.concatenate([y[x] for y in part]) for x in part[0]}
        a.check((d.own["out"], d.own["lse"]), want)
        a.lens = np.array([shared])
        want = ref.attend(dq, srows.numpy(), sscales.numpy(), [0], [shared], [0, R], T, heads, code,
                          D ** -0.5, (d.own["out"].cpu().double().numpy(),
                                      d.own["lse"].cpu().double().numpy()))
        a.check((d.out["out"], d.out["lse"]), want)
    # joined in place, over the attention of the requests' own tokens
    got = d.cache.attend_prefix(d.fmt, d.rows, d.shared_scales, d.q, d.prefix, d.prefix_len, d.starts,
                                join=d.own, out=d.own)
    torch.cuda.synchronize()
    assert got["out"] is d.own["out"] and torch.equal(got["out"], d.out["out"])
    assert torch.equal(got["lse"], d.out["lse"])
    assert d.cache.status() == (B.HS_OK, 0)
    d.cache.close()
