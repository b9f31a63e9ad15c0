"""The 8-bit key/value row calls on the GPU against the plain implementation
(kv_reference.py): attention within bounds that count its roundings, codes,
scales and kept positions bit for bit."""
import numpy as np
import pytest
import torch

import kv_reference as ref
import sparse_attention_kv_swap_gb300 as pkg
from sparse_attention_kv_swap_gb300 import binding as B

pytestmark = pytest.mark.gpu

CODES = {"e4m3": B.HS_KV_E4M3, "int8": B.HS_KV_INT8}
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
NAN_ROW = 0x7F  # the e4m3 NaN (a plain 127 in int8)


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)) if isinstance(x, np.ndarray) else x
    return t.to("cuda", dtype) if dtype is not None else t.cuda()


def random_codes(rng, shape, code):
    x = rng.standard_normal(shape).astype(np.float32)
    if code == "int8":
        return np.clip(np.rint(x * 40), -127, 127).astype(np.int8).view(np.uint8)
    t = torch.from_numpy(x * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
    return t.view(torch.uint8).numpy()


class Attend:
    """Inputs of one hs_attend call; rows that no entry refers to hold NaN codes."""

    def __init__(self, rng, B_, S, K, heads, G, D, T, code, dtype, L=None, R=None, pad=0,
                 holes=0.1, N=None):
        self.heads, self.G, self.D, self.T, self.code, self.dtype = heads, G, D, T, code, dtype
        self.L = L or max(2 * K, 40)
        self.R = R or B_ + 1
        W = 2 * heads * D + pad
        self.N = N or B_ * max(K, 1) + 7
        self.fmt = pkg.make_kv_format(heads, D, T, CODES[code], W)
        self.q = torch.from_numpy(rng.standard_normal((B_, S, heads * G, D))).to(DTYPES[dtype])
        self.req = rng.permutation(self.R)[:B_].astype(np.int32)
        self.topk = np.zeros((B_, S, K), np.int32)
        self.locs = np.zeros((B_, S, K), np.int32)
        for b in range(B_):
            for s in range(S):
                self.topk[b, s] = rng.permutation(self.L)[:K]
                self.locs[b, s] = rng.permutation(self.N)[:K]
        gone = rng.random((B_, S, K)) < holes
        self.locs[gone] = -1
        self.rows = np.full((self.N, W), NAN_ROW, np.uint8)
        used = np.unique(self.locs[self.locs >= 0])
        self.rows[used, :2 * heads * D] = random_codes(rng, (used.size, 2 * heads * D), code)
        shape = self.fmt.scales_shape(self.R, self.L)
        if code == "e4m3":
            self.scales = np.exp2(rng.integers(-9, -5, shape)).astype(np.float32)
        else:
            self.scales = (rng.random(shape) * 0.05 + 0.01).astype(np.float32)
        self.sm_scale = D ** -0.5

    def reference(self):
        return ref.attend(self.q.double().numpy(), self.rows, self.locs, self.topk, self.req,
                          self.scales, self.T, self.L, self.heads, self.code, self.sm_scale)

    def run(self, q=None, out=None, acc=None, workspace=None, stream=None, weights=True):
        q = dev(self.q) if q is None else q
        B_, S, K = self.topk.shape
        out = torch.full_like(q, float("nan")) if out is None else out
        lse = torch.full(q.shape[:3], float("nan"), device="cuda")
        w = torch.full((B_, S, K), float("nan"), device="cuda") if weights else None
        pkg.hs_attend(self.fmt, q, dev(self.rows), dev(self.locs), dev(self.topk), dev(self.req),
                      dev(self.scales), self.L, out, lse=lse, weights=w, acc=acc,
                      sm_scale=self.sm_scale, workspace=workspace, stream=stream)
        torch.cuda.synchronize()
        return out, lse, w

    def check(self, got, want=None):
        """Bounds: u is half a step of the output type; p carries f16's half step 2^-11 (and its
        subnormal step, 2^-25 of the largest) into the product; a logit is a sum of D exact
        products, each addition off by 2^-23 at most (the tensor cores truncate), times three
        32-bit factors; exp2 and the sums add a few 2^-22 and K * 2^-24."""
        out, lse, w = got
        want = want or self.reference()
        K, Hq = self.topk.shape[2], self.heads * self.G
        dz = (self.D + 8) * 2.0 ** -23 * want["logit"] + 2.0 ** -20 + K * 2.0 ** -24
        u = torch.finfo(DTYPES[self.dtype]).eps / 2
        tol = (u * np.abs(want["out"])
               + want["spread"] * (2.0 ** -11 + 2 * dz[..., None]) * (1 + u)
               + K * 2.0 ** -24 * want["biggest"] + (2.0 ** -24 if self.dtype == "fp16" else 1e-37))
        err = np.abs(out.cpu().double().numpy() - want["out"])
        assert (err <= tol).all(), (err / tol).max()
        got_lse = lse.cpu().double().numpy()
        empty = np.isneginf(want["lse"])
        assert (np.isneginf(got_lse) == empty).all()
        bad = np.abs(np.where(empty, 0, got_lse) - np.where(empty, 0, want["lse"]))
        bound = dz + 2.0 ** -22 * np.abs(np.where(empty, 0, want["lse"]))
        assert (bad <= bound).all(), (bad / bound).max()
        if w is not None:
            err = np.abs(w.cpu().double().numpy() - want["weights"])
            rel = 2 * dz.max(axis=2, keepdims=True) + Hq * 2.0 ** -24 + 2.0 ** -21
            rel = rel + 2.0 ** -22 * np.where(empty, 0, np.abs(want["lse"])).max(axis=2,
                                                                               keepdims=True)
            assert (err <= rel * want["weights"] + 1e-36).all()


@pytest.mark.parametrize("K", [0, 1, 2, 15, 16, 17, 63, 130, 777, 2048])
def test_attend_lengths(K):
    rng = np.random.default_rng(K)
    a = Attend(rng, 2, 2, K, 2, 4, 64, 16, "e4m3", "bf16")
    a.check(a.run())


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("D", [32, 64, 96, 128, 192, 256])
@pytest.mark.parametrize("heads,G,dtype", [(2, 4, "bf16"), (1, 16, "fp16"), (3, 9, "bf16")])
def test_attend_head_sizes(code, D, heads, G, dtype):
    rng = np.random.default_rng(D + G)
    a = Attend(rng, 2, 1, 150, heads, G, D, 24, code, dtype)
    a.check(a.run())


@pytest.mark.parametrize("heads,G", [(1, 1), (1, 8), (1, 128), (5, 3), (7, 5), (8, 8), (12, 4),
                                     (20, 1), (32, 1), (64, 2), (128, 1), (2, 17)])
def test_attend_head_layouts(heads, G):
    rng = np.random.default_rng(heads * 200 + G)
    a = Attend(rng, 1, 2, 90, heads, G, 64, 7, "e4m3", "fp16")
    a.check(a.run())


@pytest.mark.parametrize("B_,S", [(1, 1), (1, 4), (3, 3), (40, 1), (64, 4)])
def test_attend_batches(B_, S):
    rng = np.random.default_rng(B_ + S)
    a = Attend(rng, B_, S, 100, 1, 4, 64, 32, "int8", "bf16")
    a.check(a.run())


def test_attend_row_width_of_the_benchmark():
    """656-byte rows: five heads of 64 and padding that is never read."""
    rng = np.random.default_rng(1)
    a = Attend(rng, 3, 2, 333, 5, 4, 64, 16, "e4m3", "bf16", pad=16)
    assert a.fmt.item_size_bytes == 656
    a.check(a.run())


def test_attend_empty_queries_and_bad_entries():
    """Queries whose entries are all masked give zeros; locations, positions and requests out
    of range are masked, wherever they point."""
    rng = np.random.default_rng(2)
    a = Attend(rng, 5, 2, 70, 2, 3, 96, 16, "e4m3", "bf16", holes=0.2)
    a.locs[0, 1] = -1
    a.locs[1, 0, ::3] = a.N
    a.locs[1, 0, 1::3] = np.iinfo(np.int32).max
    a.locs[1, 1, ::2] = np.iinfo(np.int32).min
    a.topk[2, 0, ::2] = -1
    a.topk[2, 1, ::2] = a.L
    a.topk[2, 1, 1] = np.iinfo(np.int32).max
    a.req[3], a.req[4] = -1, a.R
    got = a.run()
    a.check(got)
    out, lse, w = (x.cpu().float() for x in got)
    for b, s in ((0, 1), (3, 0), (3, 1), (4, 0), (4, 1)):
        assert (out[b, s] == 0).all() and torch.isneginf(lse[b, s]).all() and (w[b, s] == 0).all()
    assert torch.isfinite(out).all()


def test_attend_one_entry_and_duplicates():
    rng = np.random.default_rng(3)
    a = Attend(rng, 2, 1, 40, 2, 4, 64, 16, "e4m3", "bf16", holes=0)
    a.locs[0, 0, :] = -1
    a.locs[0, 0, 33] = 5
    a.rows[5, :256] = random_codes(rng, 256, "e4m3")
    a.topk[1, 0, 20:] = a.topk[1, 0, :20]
    a.locs[1, 0, 20:] = a.locs[1, 0, :20]
    out, lse, w = got = a.run()
    a.check(got)
    assert abs(float(w[0, 0, 33]) - 8) < 1e-5 and float(w[0, 0].sum()) == float(w[0, 0, 33])


def test_attend_large_logits_and_scales():
    """Logits of hundreds, V scales that differ by 2^12 and a scale of zero."""
    rng = np.random.default_rng(4)
    a = Attend(rng, 2, 1, 300, 2, 8, 128, 8, "e4m3", "bf16")
    a.q = a.q * 60
    a.scales[:, :, 1] = np.exp2(rng.integers(-12, 1, a.scales[:, :, 1].shape))
    a.scales[:, ::5, 1] = 0
    a.scales[:, ::7, 0] = 0
    a.check(a.run())


def test_attend_query_magnitudes():
    """bf16 queries far outside f16's range, tiny ones and zeros."""
    rng = np.random.default_rng(5)
    a = Attend(rng, 1, 1, 64, 1, 4, 64, 16, "e4m3", "bf16")
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


def test_attend_nan_stays_in_its_head():
    """A NaN or infinite query spoils its own head; a NaN code that is selected spoils the heads
    that read it; nothing else changes."""
    rng = np.random.default_rng(6)
    a = Attend(rng, 2, 1, 50, 2, 4, 64, 16, "e4m3", "bf16", holes=0)
    clean = a.run()
    a.q[0, 0, 1, 3] = float("nan")
    a.q[0, 0, 6, 3] = float("inf")
    out, lse, _ = a.run()
    assert torch.isnan(out[0, 0, 1]).all() and torch.isnan(lse[0, 0, 1])
    assert torch.isnan(out[0, 0, 6]).any()
    for i in (0, 2, 3, 4, 5, 7):
        assert torch.equal(out[0, 0, i], clean[0][0, 0, i])
    assert torch.equal(out[1], clean[0][1])
    a.q[0, 0, 1, 3], a.q[0, 0, 6, 3] = 0, 0
    a.rows[a.locs[1, 0, 7], 64 + 5] = NAN_ROW  # K of head 1
    out, lse, _ = a.run()
    assert torch.isnan(out[1, 0, 4:]).all() and torch.equal(out[1, 0, :4], clean[0][1, 0, :4])


def test_attend_strides_and_alignment():
    """Queries and outputs inside larger tensors, transposed, and off 16-byte alignment."""
    rng = np.random.default_rng(7)
    a = Attend(rng, 3, 2, 60, 2, 2, 64, 16, "e4m3", "fp16")
    want = a.reference()
    plain = a.run()
    wide = torch.zeros((3, 2, 6, 80), dtype=torch.float16, device="cuda")
    for off in (0, 1, 8):
        q = wide[:, :, 1:5, off:off + 64]
        q.copy_(a.q)
        out = torch.zeros((4, 2, 3, 100), dtype=torch.float16, device="cuda").permute(2, 1, 0, 3)
        view = out[..., off:off + 64]
        got = a.run(q=q, out=view)
        a.check(got, want)
        assert torch.equal(got[0], plain[0])
        assert (out[..., :off] == 0).all() and (out[..., off + 64:] == 0).all()
    one = dev(a.q)[:, :, :1].expand(3, 2, 4, 64)  # a broadcast query (stride 0)
    a.q = one.cpu().contiguous()
    a.check(a.run(q=one))


@pytest.mark.parametrize("S", [1, 3])
def test_attend_accumulates_weights(S):
    rng = np.random.default_rng(8 + S)
    a = Attend(rng, 4, S, 200, 2, 4, 64, 16, "e4m3", "bf16", L=260)
    start = rng.random((a.R, a.L)).astype(np.float32)
    acc = dev(start)
    out, lse, w = a.run(acc=acc)
    want = start.copy()
    w = w.cpu().numpy()
    for b in range(4):
        for s in range(S):
            np.add.at(want[a.req[b]], a.topk[b, s], w[b, s])
    assert np.array_equal(acc.cpu().numpy(), want)
    if S == 1:  # without a weights output too
        acc = dev(start)
        a.run(acc=acc, weights=False)
        assert np.array_equal(acc.cpu().numpy(), want)


@pytest.mark.parametrize("code,heads,G,D,K", [("e4m3", 8, 8, 128, 14000), ("int8", 2, 40, 256, 9000),
                                              ("e4m3", 1, 4, 64, 50000), ("e4m3", 8, 8, 128, 20000),
                                              ("int8", 3, 24, 256, 18000)])
def test_attend_longer_than_shared_memory(code, heads, G, D, K):
    """Selections whose scores go through the workspace, and long ones that fit an SM's tensor
    memory (65536 scores in each of 16 CTAs)."""
    rng = np.random.default_rng(K)
    a = Attend(rng, 1, 1, K, heads, G, D, 64, code, "bf16")
    n = pkg.hs_attend_workspace_bytes(a.fmt, 1, 1, K, heads * G)
    assert (n > 0) == (heads * G * K > 1 << 20)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    a.check(a.run(workspace=ws))


def test_attend_rows_past_4_gb():
    """Rows whose byte offsets pass 32 bits."""
    rng = np.random.default_rng(9)
    heads, G, D, K = 8, 2, 128, 96
    n = (5 << 30) // 2048
    a = Attend(rng, 1, 1, K, heads, G, D, 64, "e4m3", "bf16", holes=0)
    big = torch.full((n, 2048), NAN_ROW, dtype=torch.uint8, device="cuda")
    far = (n - 1 - rng.permutation(n // 2)[:K]).astype(np.int32)
    big[torch.from_numpy(far).cuda().long()] = dev(a.rows)[dev(a.locs[0, 0]).long()]
    out, lse, _ = a.run()
    locs = dev(far.reshape(1, 1, K))
    got = torch.empty_like(out)
    got_lse = torch.empty_like(lse)
    pkg.hs_attend(a.fmt, dev(a.q), big, locs, dev(a.topk), dev(a.req), dev(a.scales), a.L, got,
                  lse=got_lse, sm_scale=a.sm_scale)
    torch.cuda.synchronize()
    assert torch.equal(got, out) and torch.equal(got_lse, lse)


def test_attend_repeats_streams_and_graphs():
    """The same bits on every run, on another stream and replayed from a CUDA graph."""
    rng = np.random.default_rng(10)
    a = Attend(rng, 6, 4, 500, 3, 5, 96, 32, "int8", "fp16", L=900)
    q, rows, locs, topk = dev(a.q), dev(a.rows), dev(a.locs), dev(a.topk)
    req, scales = dev(a.req), dev(a.scales)

    def buffers():
        return (torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda"),
                torch.zeros(topk.shape, device="cuda"), torch.zeros((a.R, a.L), device="cuda"))

    def call(o, stream=None):
        pkg.hs_attend(a.fmt, q, rows, locs, topk, req, scales, a.L, o[0], lse=o[1], weights=o[2],
                      acc=o[3], stream=stream)

    first = buffers()
    call(first)
    torch.cuda.synchronize()
    again = buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(again, stream=side)
    side.synchronize()
    for x, y in zip(first, again):
        assert torch.equal(x, y)
    held = buffers()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(held)
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(first, held):
        assert torch.equal(x, y)


# ---- quantisation ---------------------------------------------------------------

def quantize_case(rng, B_, M, heads, D, T, code, dtype, L, start=None, count=None, pad=0,
                  pinned=False):
    fmt = pkg.make_kv_format(heads, D, T, CODES[code], 2 * heads * D + pad)
    R = B_ + 2
    size = np.exp(rng.standard_normal((1, 1, heads, D)))
    k = torch.from_numpy(rng.standard_normal((B_, M, heads, D)) * size).to(DTYPES[dtype])
    v = torch.from_numpy(rng.standard_normal((B_, M, heads, D))).to(DTYPES[dtype])
    rows = torch.from_numpy(rng.integers(0, 256, (R, L, fmt.item_size_bytes)).astype(np.uint8))
    rows[..., :2 * heads * D] = torch.from_numpy(random_codes(rng, (R, L, 2 * heads * D), code))
    shape = fmt.scales_shape(R, L)
    if code == "e4m3":
        scales = torch.from_numpy(np.exp2(rng.integers(-9, -4, shape)).astype(np.float32))
    else:
        scales = torch.from_numpy((rng.random(shape) * 0.05).astype(np.float32))
    req = rng.permutation(R)[:B_].astype(np.int32)
    count = rng.integers(0, M + 1, B_) if count is None else np.asarray(count)
    start = rng.integers(0, L - count + 1) if start is None else np.asarray(start)
    return fmt, k, v, req, start.astype(np.int32), count.astype(np.int32), rows, scales


def run_quantize(case, code):
    fmt, k, v, req, start, count, rows, scales = case
    drows, dscales = dev(rows), dev(scales)
    pkg.hs_quantize_kv(fmt, dev(k), dev(v), dev(req), dev(start), dev(count), drows, dscales)
    torch.cuda.synchronize()
    ref.quantize(k, v, req, start, count, rows, scales, fmt.block_tokens, code)
    assert torch.equal(dscales.cpu(), scales)
    assert torch.equal(drows.cpu(), rows)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D,T,M", [(64, 16, 1), (32, 1, 5), (96, 48, 130), (128, 64, 200),
                                   (256, 256, 300), (192, 700, 900)])
def test_quantize(code, dtype, D, T, M):
    rng = np.random.default_rng(D + T + M)
    run_quantize(quantize_case(rng, 5, M, 3, D, T, code, dtype, L=M + 333, pad=16), code)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_quantize_grows_a_filling_block(code):
    """Tokens one by one into one block, each larger than the last: the scale grows, the older
    codes are rounded again; then smaller ones, which leave it."""
    rng = np.random.default_rng(11)
    heads, D, T, L = 2, 64, 16, 64
    fmt = pkg.make_kv_format(heads, D, T, CODES[code])
    rows = torch.zeros((2, L, 256), dtype=torch.uint8)
    scales = torch.full(fmt.scales_shape(2, L), 7.0)  # of the slot's previous user
    drows, dscales = dev(rows), dev(scales)
    for t in range(40):
        f = 1.7 ** (t % T) if t < 2 * T else 0.3
        k = torch.from_numpy(rng.standard_normal((1, 1, heads, D)) * f).bfloat16()
        v = torch.from_numpy(rng.standard_normal((1, 1, heads, D)) / f).bfloat16()
        req, start, one = np.array([1]), np.array([t]), np.array([1])
        pkg.hs_quantize_kv(fmt, dev(k), dev(v), dev(req, torch.int32), dev(start, torch.int32),
                           dev(one, torch.int32), drows, dscales)
        torch.cuda.synchronize()
        ref.quantize(k, v, req, start, one, rows, scales, T, code)
        assert torch.equal(dscales.cpu(), scales) and torch.equal(drows.cpu(), rows), t
    assert (scales[1, :3] != 7.0).all() and (scales[1, 3:] == 7.0).all()


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_quantize_special_values(code):
    """Zeros, infinities, NaN, the smallest and the largest magnitudes."""
    rng = np.random.default_rng(12)
    case = quantize_case(rng, 8, 32, 1, 64, 16, code, "fp32", L=64, start=[0] * 8,
                         count=[32] * 8)
    k = case[1]
    k[0] = 0
    k[1, :, 0, 5] = float("inf")
    k[2, 3, 0, 7] = float("nan")
    k[3] *= 1e-35
    k[4] *= 1e-42
    k[5] *= 1e37
    k[6, :16] = -448.0
    k[7, 0, 0, 0] = float("-inf")
    k[7, :, 0, 1] = 3.4e38
    run_quantize(case, code)


def test_quantize_skips_bad_entries():
    rng = np.random.default_rng(13)
    case = quantize_case(rng, 7, 10, 2, 32, 4, "e4m3", "bf16", L=50,
                         start=[-1, 45, 0, 2147483647, 3, 0, 41], count=[4, 6, 11, 10, 0, -3, 9])
    req = case[3]
    req[6] = 99
    run_quantize(case, "e4m3")


def test_quantize_strides_and_pinned_rows():
    """K and V as slices of one projection, transposed and broadcast inputs, odd alignment,
    and rows in pinned host memory."""
    rng = np.random.default_rng(14)
    code, heads, D, T, M = "e4m3", 2, 64, 16, 40
    for kind in ("slice", "transposed", "broadcast", "odd"):
        case = list(quantize_case(rng, 3, M, heads, D, T, code, "bf16", L=100))
        fmt, k, v, req, start, count, rows, scales = case
        if kind == "slice":
            both = dev(torch.cat((k, v), dim=-1))
            dk, dv = both[..., :D], both[..., D:]
        elif kind == "transposed":
            dk = dev(k).permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3)
            dv = dev(v).transpose(0, 1).contiguous().transpose(0, 1)
        elif kind == "broadcast":
            k, v = k[:, :, :1].expand_as(k), v[:1].expand_as(v)
            dk, dv = dev(k.contiguous())[:, :, :1].expand_as(k), dev(v[:1].contiguous()).expand_as(v)
        else:
            flat = torch.zeros(k.numel() + 1, dtype=k.dtype, device="cuda")
            dk = flat[1:].view(k.shape)
            dk.copy_(k)
            dv = dev(v)
        pinned = rows.clone().pin_memory()
        dscales = dev(scales)
        pkg.hs_quantize_kv(fmt, dk, dv, dev(req), dev(start), dev(count), pinned, dscales)
        torch.cuda.synchronize()
        ref.quantize(k, v, req, start, count, rows, scales, T, code)
        assert torch.equal(dscales.cpu(), scales) and torch.equal(pinned, rows), kind


@pytest.mark.parametrize("dense", [False, True], ids=["hash", "dense"])
@pytest.mark.parametrize("T,E", [(8, 16), (24, 10), (16, 0)])
def test_append_keeps_every_copy_equal(dense, T, E):
    """Decode steps through a swap-in handle: after each write-back every location that a
    swap-in returns, hot row, extra page or fresh copy, holds the host row, and that is what
    the plain implementation writes."""
    from sparse_attention_kv_swap_gb300.cache import SwapInCache
    rng = np.random.default_rng(15 + T)
    R, L, H, K, S, heads, D = 4, 200, 24, 12, 2, 5, 64
    cfg = pkg.make_config(R, L, 656, H, K, S, index_kind=int(dense), extra_page_size=E)
    fmt = pkg.make_kv_format(heads, D, T, B.HS_KV_E4M3, 656)
    cache = SwapInCache(cfg)
    cache.host_pools[0].random_(0, 120)
    rows = cache.host_pools[0].clone()
    scales = torch.zeros(fmt.scales_shape(R, L))
    dscales = dev(scales)
    n = np.zeros(R, np.int64)
    for step in range(14):
        B_ = int(rng.integers(1, R + 1))
        req = rng.permutation(R)[:B_].astype(np.int32)
        M = 30 if step == 0 else int(rng.integers(1, 4))
        if step == 0:
            req, B_ = np.arange(R, dtype=np.int32), R
        count = rng.integers(1, M + 1, B_).astype(np.int32)
        start = n[req].astype(np.int32)
        f = np.exp(rng.standard_normal((B_, M, 1, 1)))
        k = torch.from_numpy(rng.standard_normal((B_, M, heads, D)) * f).bfloat16()
        v = torch.from_numpy(rng.standard_normal((B_, M, heads, D)) * f).bfloat16()
        cache.append_kv(fmt, dscales, dev(k), dev(v), dev(req), dev(start), dev(count))
        torch.cuda.synchronize()
        ref.quantize(k, v, req, start, count, rows, scales, T, "e4m3")
        assert torch.equal(dscales.cpu(), scales)
        assert torch.equal(cache.host_pools[0], rows)
        n[req] = start + count
        every = np.arange(R, dtype=np.int32)
        topk = np.stack([[rng.permutation(int(n[q]))[:K] if n[q] >= K else
                          np.arange(K) for _ in range(S)] for q in every]).astype(np.int32)
        topk[:, 0, 0] = n - 1
        locs = cache.swap_in(dev(every), dev(n.astype(np.int32)), dev(topk))["device_locs"].cpu()
        got = cache.device_kv[0].cpu()
        for q in range(R):
            for s in range(S):
                for j in range(K):
                    t = int(topk[q, s, j])
                    if t < n[q]:  # keys and values; the padding is not the call's to write
                        row = got[int(locs[q, s, j]), :2 * heads * D]
                        assert torch.equal(row, rows[q, t, :2 * heads * D]), (step, q, t)
    assert cache.status() == (B.HS_OK, 0)
    bad = dev(np.array([99], np.int32))
    one = dev(np.array([1], np.int32))
    cache.append_kv(fmt, dscales, dev(k[:1]), dev(v[:1]), bad, one, one)
    rc, flags = cache.status()
    assert rc == B.HS_ERR_DEVICE_STATUS and flags == B.HS_STATUS_BAD_APPEND
    cache.close()


# ---- eviction -------------------------------------------------------------------

def run_evict(acc, req, seq_lens, recent, budget, with_acc=True):
    B_ = len(req)
    keep = torch.full((B_, budget), 77, dtype=torch.int32, device="cuda")
    kept = torch.full((B_,), 77, dtype=torch.int32, device="cuda")
    ka = torch.full((B_, budget), 77.0, device="cuda") if with_acc else None
    pkg.hs_evict(dev(acc), dev(np.asarray(req, np.int32)), dev(np.asarray(seq_lens, np.int32)),
                 recent, keep, kept, ka)
    torch.cuda.synchronize()
    wk, wn, wa = ref.evict(acc, req, seq_lens, recent, budget)
    assert np.array_equal(kept.cpu().numpy(), wn)
    assert np.array_equal(keep.cpu().numpy(), wk)
    if with_acc:
        assert np.array_equal(ka.cpu().numpy(), wa, equal_nan=True)


@pytest.mark.parametrize("L,budget,recent", [(1, 1, 0), (2, 1, 0), (2, 1, 1), (33, 32, 5),
                                             (500, 100, 100), (500, 499, 3), (4096, 2048, 256),
                                             (8193, 17, 0), (20000, 15000, 1), (131072, 9999, 777)])
def test_evict(L, budget, recent):
    rng = np.random.default_rng(L)
    acc = np.exp(3 * rng.standard_normal((4, L))).astype(np.float32)
    run_evict(acc, [2, 0, 3], [L, max(L - 7, 0), L + 5], recent, budget)


def test_evict_ties_and_special_weights():
    """Equal weights go to the lowest positions; zeros of both signs are equal; negative,
    infinite and NaN weights have their places."""
    rng = np.random.default_rng(16)
    L = 9000
    acc = rng.integers(0, 3, (6, L)).astype(np.float32)
    acc[1] = 1.0
    acc[2] = np.where(rng.random(L) < 0.5, 0.0, -0.0)
    acc[3] = rng.standard_normal(L)
    acc[3, rng.integers(0, L, 50)] = np.nan
    acc[3, rng.integers(0, L, 50)] = np.inf
    acc[3, rng.integers(0, L, 50)] = -np.inf
    acc[4] = np.nan
    acc[5] = np.exp2(rng.integers(-149, 127, L).astype(np.float64)).astype(np.float32)
    for budget, recent in ((3000, 100), (8990, 0), (1, 0)):
        run_evict(acc, np.arange(6), [L] * 6, recent, budget)


def test_evict_lengths_and_bad_requests():
    rng = np.random.default_rng(17)
    acc = rng.random((3, 300)).astype(np.float32)
    run_evict(acc, [0, 1, 2, -1, 3, 0], [0, -4, 50, 300, 300, 51], 10, 50)
    run_evict(acc, [0, 1, 2], [300, 299, 51], 50, 50, with_acc=False)


def test_accumulate():
    rng = np.random.default_rng(18)
    B_, S, K, R, L = 5, 4, 1500, 6, 3000
    topk = np.stack([[rng.permutation(L + 40)[:K] - 20 for _ in range(S)] for _ in range(B_)])
    topk = topk.astype(np.int32)
    w = rng.random((B_, S, K)).astype(np.float32)
    req = np.array([4, 0, 6, 2, -1], np.int32)
    counts = np.array([4, 1, 2, 0, 3], np.int32)
    for n in (None, counts):
        acc = rng.random((R, L)).astype(np.float32)
        got = dev(acc)
        pkg.hs_accumulate(dev(w), dev(topk), dev(req), got, None if n is None else dev(n))
        torch.cuda.synchronize()
        for b in range(B_):
            if 0 <= req[b] < R:
                for s in range(S if n is None else n[b]):
                    ok = (topk[b, s] >= 0) & (topk[b, s] < L)
                    acc[req[b], topk[b, s][ok]] += w[b, s][ok]
        assert np.array_equal(got.cpu().numpy(), acc)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("D,T,budget", [(64, 16, 100), (96, 48, 333), (128, 64, 64), (256, 256, 300),
                                        (192, 700, 650), (32, 1, 9)])
def test_compact(code, D, T, budget):
    rng = np.random.default_rng(D + T)
    heads, sR, sL, dR, dL = 3, 4, 900, 5, budget + 11
    fmt = pkg.make_kv_format(heads, D, T, CODES[code], 2 * heads * D + 32)
    src = torch.from_numpy(rng.integers(0, 256, (sR, sL, fmt.item_size_bytes)).astype(np.uint8))
    src[..., :2 * heads * D] = torch.from_numpy(random_codes(rng, (sR, sL, 2 * heads * D), code))
    shape = fmt.scales_shape(sR, sL)
    if code == "e4m3":
        ss = torch.from_numpy(np.exp2(rng.integers(-12, -4, shape)).astype(np.float32))
    else:
        ss = torch.from_numpy((rng.random(shape) * 0.05).astype(np.float32))
    ss[1, ::3] = 0
    dst = torch.from_numpy(rng.integers(0, 256, (dR, dL, fmt.item_size_bytes)).astype(np.uint8))
    ds = torch.full(fmt.scales_shape(dR, dL), 3.0)
    B_ = 5
    keep = np.stack([np.sort(rng.permutation(sL)[:budget]) for _ in range(B_)]).astype(np.int32)
    keep[2, 1] = -1
    keep[2, 2] = sL
    kept = torch.tensor([budget, budget // 2, budget + 9, 0, budget], dtype=torch.int32)
    sq = torch.tensor([1, 0, 3, 2, 4], dtype=torch.int32)  # the last one is out of range
    dq = torch.tensor([4, 2, 0, 1, 3], dtype=torch.int32)
    keep = torch.from_numpy(keep)
    gd, gs = dev(dst), dev(ds)
    pkg.hs_compact_kv(fmt, dev(src), dev(ss), dev(sq), dev(keep), dev(kept), gd, gs, dev(dq))
    torch.cuda.synchronize()
    ref.compact(src, ss, sq, keep, kept, dst, ds, dq, T, heads, D, code)
    assert torch.equal(gs.cpu(), ds)
    assert torch.equal(gd.cpu(), dst)


def test_cache_evict_shrinks_every_layer():
    """SwapInCache.evict: the kept rows move to the first positions of the host pool, scales
    and sums follow, and swap-ins of the shortened sequences return them."""
    from sparse_attention_kv_swap_gb300.cache import SwapInCache
    rng = np.random.default_rng(19)
    R, L, H, K, layers, heads, D, T, E = 3, 120, 40, 30, 2, 2, 64, 16, 16
    cfg = pkg.make_config(R, L, 256, H, K, 1, num_layers=layers, extra_page_size=E)
    fmt = pkg.make_kv_format(heads, D, T)
    cache = SwapInCache(cfg)
    scales = [torch.zeros(fmt.scales_shape(R, L), device="cuda") for _ in range(layers)]
    acc = [dev(rng.random((R, L)).astype(np.float32)) for _ in range(layers)]
    every = dev(np.arange(R, dtype=np.int32))
    lens = np.array([120, 75, 40])
    for l in range(layers):
        kv = torch.from_numpy(rng.standard_normal((R, L, heads, D))).bfloat16()
        cache.append_kv(fmt, scales[l], dev(kv), dev(kv.flip(1)), every, torch.zeros_like(every),
                        dev(lens.astype(np.int32)), layer_id=l)
        topk = dev(np.stack([[rng.permutation(40)[:K]] for _ in range(R)]).astype(np.int32))
        cache.swap_in(every, dev(lens.astype(np.int32)), topk, l)
    torch.cuda.synchronize()
    pools = [p.clone() for p in cache.host_pools]
    was = [s.cpu() for s in scales]
    sums = [x.cpu().numpy() for x in acc]
    budget, recent = 50, 10
    gone = [0, 1]
    n = cache.evict(fmt, scales, acc, gone, lens[gone].tolist(), budget, recent)
    assert n == [50, 50]
    torch.cuda.synchronize()
    new_lens = np.array([50, 50, 40], np.int32)
    for l in range(layers):
        keep, kept, ka = ref.evict(sums[l], gone, lens[gone], recent, budget)
        want, ws = pools[l].clone(), was[l].clone()
        dst, ds = torch.zeros((2, budget, 256), dtype=torch.uint8), torch.zeros((2, 4, 2, heads))
        ref.compact(pools[l], was[l], gone, torch.from_numpy(keep), torch.from_numpy(kept), dst,
                    ds, [0, 1], T, heads, D, "e4m3")
        want[gone, :budget] = dst
        ws[gone, :4] = ds
        assert torch.equal(cache.host_pools[l], want)
        assert torch.equal(scales[l].cpu()[:, :4], ws[:, :4])
        got = acc[l].cpu().numpy()
        assert np.array_equal(got[gone, :budget], ka) and (got[gone, budget:] == 0).all()
        assert np.array_equal(got[2], sums[l][2])
        topk = np.stack([[rng.permutation(40)[:K]] for _ in range(R)]).astype(np.int32)
        topk[:, 0, 0] = new_lens - 1
        locs = cache.swap_in(every, dev(new_lens), dev(topk), l)["device_locs"].cpu()
        rows = cache.device_kv[l].cpu()
        for q in range(R):
            for j in range(K):
                assert torch.equal(rows[int(locs[q, 0, j])], want[q, int(topk[q, 0, j])])
    assert cache.status() == (B.HS_OK, 0)
    cache.close()


# ---- longer and chained calls ---------------------------------------------------

@pytest.mark.parametrize("L,budget,recent", [(131073, 1000, 10), (300001, 70000, 4096)])
def test_evict_longer_than_the_registers_hold(L, budget, recent):
    rng = np.random.default_rng(L)
    acc = np.exp(2 * rng.standard_normal((2, L))).astype(np.float32)
    acc[1] = rng.integers(0, 50, L)
    run_evict(acc, [1, 0], [L, L - 1], recent, budget)


@pytest.mark.parametrize("requests,L", [(1, 9000), (200, 9000), (40, 20000), (3, 40000), (90, 40000),
                                        (160, 70000)])
def test_evict_many_requests(requests, L):
    rng = np.random.default_rng(requests + L)
    acc = np.exp(2 * rng.standard_normal((5, L))).astype(np.float32)
    acc[3] = rng.integers(0, 5, L)
    seq = L - rng.integers(0, L // 2, requests)
    run_evict(acc, rng.integers(0, 5, requests), seq, 100, L // 3)


@pytest.mark.parametrize("S,K", [(1, 9001), (4, 8193), (5, 600), (7, 8200), (2, 1), (4, 8192)])
def test_accumulate_steps_and_lengths(S, K):
    rng = np.random.default_rng(100 * S + K)
    R, L = 3, K + 33
    topk = np.stack([[rng.permutation(L)[:K] for _ in range(S)] for _ in range(2)])
    topk = topk.astype(np.int32)
    w = rng.random((2, S, K)).astype(np.float32)
    acc = rng.random((R, L)).astype(np.float32)
    got = dev(acc)
    pkg.hs_accumulate(dev(w), dev(topk), dev(np.array([2, 0], np.int32)), got)
    torch.cuda.synchronize()
    for b, q in enumerate((2, 0)):
        for s in range(S):
            acc[q, topk[b, s]] += w[b, s]
    assert np.array_equal(got.cpu().numpy(), acc)


def test_calls_follow_one_another():
    """Calls whose inputs the call before them writes, directly and from a graph: positions kept
    by an eviction are what the next accumulation adds to and the next compaction copies."""
    rng = np.random.default_rng(21)
    B_, L, budget, recent, heads, D, T = 48, 3000, 700, 50, 3, 64, 32
    fmt = pkg.make_kv_format(heads, D, T, B.HS_KV_INT8)
    k = torch.from_numpy(rng.standard_normal((B_, L, heads, D))).bfloat16()
    v = torch.from_numpy(rng.standard_normal((B_, L, heads, D))).bfloat16()
    first = rng.random((B_, L)).astype(np.float32)
    more = rng.random((B_, 1, budget)).astype(np.float32)
    req = np.arange(B_, dtype=np.int32)
    dk, dv, dmore, dreq = dev(k), dev(v), dev(more), dev(req)
    zero, n = torch.zeros_like(dreq), torch.full_like(dreq, L)
    rows = torch.zeros((B_, L, 2 * heads * D), dtype=torch.uint8, device="cuda")
    scales = torch.zeros(fmt.scales_shape(B_, L), device="cuda")
    acc = dev(first)
    keep = torch.empty((2, B_, 1, budget), dtype=torch.int32, device="cuda")
    kept = torch.empty((2, B_), dtype=torch.int32, device="cuda")
    dst = torch.zeros((B_, budget, 2 * heads * D), dtype=torch.uint8, device="cuda")
    ds = torch.zeros(fmt.scales_shape(B_, budget), device="cuda")

    def calls():
        acc.copy_(dfirst)
        pkg.hs_quantize_kv(fmt, dk, dv, dreq, zero, n, rows, scales)
        pkg.hs_evict(acc, dreq, n, recent, keep[0, :, 0], kept[0])
        pkg.hs_accumulate(dmore, keep[0], dreq, acc)
        pkg.hs_evict(acc, dreq, n, recent, keep[1, :, 0], kept[1])
        pkg.hs_compact_kv(fmt, rows, scales, dreq, keep[1, :, 0], kept[1], dst, ds, dreq)

    dfirst = dev(first)
    wr, ws = torch.zeros_like(rows, device="cpu"), torch.zeros_like(scales, device="cpu")
    ref.quantize(k, v, req, [0] * B_, [L] * B_, wr, ws, T, "int8")
    one, count, _ = ref.evict(first, req, [L] * B_, recent, budget)
    sums = first.copy()
    for b in range(B_):
        sums[b, one[b]] += more[b, 0]
    two, count, _ = ref.evict(sums, req, [L] * B_, recent, budget)
    wd, wds = torch.zeros_like(dst, device="cpu"), torch.zeros_like(ds, device="cpu")
    ref.compact(wr, ws, req, torch.from_numpy(two), torch.from_numpy(count), wd, wds, req, T, heads,
                D, "int8")

    def check():
        torch.cuda.synchronize()
        assert torch.equal(rows.cpu(), wr) and torch.equal(scales.cpu(), ws)
        assert np.array_equal(keep[0, :, 0].cpu().numpy(), one)
        assert np.array_equal(acc.cpu().numpy(), sums)
        assert np.array_equal(keep[1, :, 0].cpu().numpy(), two)
        assert torch.equal(ds.cpu(), wds) and torch.equal(dst.cpu(), wd)

    for _ in range(3):
        calls()
        check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for x in (rows, scales, acc, keep, kept, dst, ds):
        x.zero_()
    for _ in range(3):
        graph.replay()
    check()


@pytest.mark.parametrize("code,dtype,heads,group,D,T", [("e4m3", "bf16", 2, 4, 64, 16),
                                                        ("int8", "fp16", 3, 2, 96, 24)])
def test_decode_example(code, dtype, heads, group, D, T):
    """The example's loop, eviction in between: codes and scales bit for bit, every step's
    attention within its bounds, over the rows that the host pool should hold."""
    import importlib.util
    import pathlib
    path = pathlib.Path(__file__).resolve().parent.parent / "examples" / "decode_8bit.py"
    spec = importlib.util.spec_from_file_location("decode_8bit", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    rng = np.random.default_rng(22)
    R, limit, budget, recent, top_k = 3, 100, 41, 7, 30
    d = example.Decoder(R, limit, budget, recent, top_k, 2 * top_k, heads, group, D, T, CODES[code],
                        DTYPES[dtype])
    pool = d.cache.host_pools[0]
    pool.zero_()
    rows, scales = pool.clone(), torch.zeros_like(d.scales, device="cpu")
    acc = np.zeros((R, limit), np.float32)
    req = np.arange(R, dtype=np.int32)

    def rand(*shape):
        return torch.from_numpy(rng.standard_normal(shape)).to(DTYPES[dtype])

    lens = np.array([95, 60, 97])
    k, v = rand(R, 97, heads, D), rand(R, 97, heads, D)
    d.prompt(dev(k), dev(v), lens)
    ref.quantize(k, v, req, [0] * R, lens, rows, scales, T, code)
    cut = 0
    for step in range(90):
        torch.cuda.synchronize()
        full = [i for i in range(R) if lens[i] == limit]
        if full:
            keep, kept, ka = ref.evict(acc, full, lens[full], recent, budget)
            nb = d.fmt.num_blocks(budget)
            dst = torch.zeros((len(full), budget, rows.shape[2]), dtype=torch.uint8)
            ds = torch.zeros((len(full), nb, 2, heads))
            ref.compact(rows, scales, full, torch.from_numpy(keep), torch.from_numpy(kept), dst, ds,
                        list(range(len(full))), T, heads, D, code)
            rows[full, :budget], scales[full, :nb] = dst, ds
            acc[full], lens[full] = 0, budget
            acc[full, :budget] = ka
            cut += len(full)
        assert d.make_room() == full
        q, k, v = rand(R, 1, heads * group, D), rand(R, 1, heads, D), rand(R, 1, heads, D)
        topk = d.select()
        d.step(dev(q), dev(k), dev(v), topk)
        torch.cuda.synchronize()
        ref.quantize(k, v, req, lens, [1] * R, rows, scales, T, code)
        lens += 1
        assert torch.equal(pool, rows) and torch.equal(d.scales.cpu(), scales), step
        topk = topk.cpu().numpy()
        assert (topk[:, 0, 0] == lens - 1).all()
        a = Attend.__new__(Attend)
        a.heads, a.G, a.D, a.T, a.code, a.dtype, a.L = heads, group, D, T, code, dtype, limit
        a.q, a.topk, a.req, a.scales, a.sm_scale = q, topk, req, scales.numpy(), D ** -0.5
        a.rows = rows.reshape(R * limit, -1).numpy()
        a.locs = np.where(topk < 0, -1, topk + limit * req[:, None, None])
        a.check((d.out["out"], d.out["lse"], d.out["weights"]))
        w = d.out["weights"].cpu().numpy()
        for b in range(R):
            ok = topk[b, 0] >= 0
            acc[b, topk[b, 0, ok]] += w[b, 0, ok]
        assert np.array_equal(d.acc.cpu().numpy(), acc)
    assert cut == 5 and d.cache.status() == (B.HS_OK, 0)
    d.cache.close()


def test_cache_evict_refuses_before_it_acts():
    from sparse_attention_kv_swap_gb300.cache import SwapInCache
    cfg = pkg.make_config(2, 40, 256, 16, 8, 1)
    fmt = pkg.make_kv_format(2, 64, 16)
    cache = SwapInCache(cfg)
    cache.host_pools[0].random_(0, 120)
    pool = cache.host_pools[0].clone()
    scales, acc = [cache.kv_scales(fmt) + 1], [torch.ones((2, 40), device="cuda")]
    for requests, lens, budget, recent in (([0], [40], 8, 9), ([0], [40], 8, -1), ([0], [40], 0, 0),
                                           ([0, 1], [40], 8, 2), ([0], [41], 8, 2),
                                           ([0], [-1], 8, 2)):
        with pytest.raises(ValueError):
            cache.evict(fmt, scales, acc, requests, lens, budget, recent)
    assert cache.evict(fmt, scales, acc, [], [], 8, 2) == []
    assert cache.evict(fmt, scales, acc, [1], [0], 8, 2) == [0]  # nothing to keep
    torch.cuda.synchronize()
    assert torch.equal(cache.host_pools[0], pool)
    cache.close()
