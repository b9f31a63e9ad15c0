"""The calls around a decode step on the CPU: what they refuse, before any launch, at the C
entry points and in the Python binding, and the layout of the structures that cross it."""
import ctypes
import math
import re

import numpy as np
import pytest
import torch

import sparse_attention_kv_swap_gb300 as pkg
import step_reference as ref
from sparse_attention_kv_swap_gb300 import binding as B


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_kv_swap_gb300 import build
    build.build()
    return B.load_library()


# Addresses below are never dereferenced: every call is refused on the host.
OK, ODD = 0x20000, 0x20002
bad, unsupported = B.HS_ERR_INVALID_ARG, B.HS_ERR_UNSUPPORTED
STRIDES = (ctypes.c_int64 * 3)(1, 1, 1)


def test_header_constants_and_structs():
    text = open(B.HEADER).read()
    consts = dict(re.findall(r"#define (HS_MAX_[A-Z0-9_]+) +(\d+)", text))
    for name in ("HS_MAX_ROPE_AXES", "HS_MAX_SELECT_BLOCKS", "HS_MAX_SELECT_WIDTH",
                 "HS_MAX_PREFIXES"):
        assert int(consts[name]) == getattr(B, name), name
    code = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    for struct, cls, pack in (("hs_norm_rope_args", B._HsNormRopeArgs, B._NORM_ROPE_ARGS),
                              ("hs_select_args", B._HsSelectArgs, B._SELECT_ARGS),
                              ("hs_prefix_args", B._HsPrefixArgs, B._PREFIX_ARGS)):
        body = re.search(r"typedef struct %s \{(.*?)\}" % struct, code, re.S).group(1)
        names = []
        for decl in body.split(";"):
            if decl.strip():
                names += [re.findall(r"(\w+)(?:\[\d+\])?$", part.strip())[0]
                          for part in decl.split(",")]
        assert names == [n for n, _ in cls._fields_], struct
        # the packed form that the binding passes has the same layout
        fields = []
        for _, kind in cls._fields_:
            n = getattr(kind, "_length_", 1)
            fields += range(100 + len(fields), 100 + len(fields) + n)
        a = cls.from_buffer_copy(pack.pack(*fields))
        flat = []
        for name, _ in cls._fields_:
            x = getattr(a, name)
            flat += list(x) if isinstance(x, ctypes.Array) else [int(x)]
        assert flat == fields and pack.size == ctypes.sizeof(cls)


def test_norm_rope_refuses(lib):
    base = dict(q_dev=OK, k_dev=OK, q_out_dev=OK, k_out_dev=OK, dtype=B.HS_DTYPE_BF16, batch=2,
                tokens=3, num_heads=8, num_kv_heads=2, head_dim=64, rot_dim=64, adjacent=0,
                num_axes=1, eps=1e-6, q_stride=STRIDES, k_stride=STRIDES, q_out_stride=STRIDES,
                k_out_stride=STRIDES, q_weight_dev=OK, k_weight_dev=OK, pos_dev=OK, turns_dev=OK,
                axis_dev=OK, count_dev=OK)

    def call(**kw):
        return lib.hs_norm_rope(ctypes.byref(B._HsNormRopeArgs(**dict(base, **kw))), None)

    assert lib.hs_norm_rope(None, None) == bad
    for kw in (dict(batch=-1), dict(tokens=-1), dict(num_heads=-1), dict(num_kv_heads=-1),
               dict(dtype=-1), dict(dtype=3), dict(rot_dim=-16), dict(rot_dim=80),
               dict(rot_dim=24), dict(num_axes=0), dict(adjacent=2), dict(head_dim=0),
               dict(eps=0.0), dict(eps=-1.0), dict(eps=math.nan), dict(q_dev=None),
               dict(k_dev=None), dict(q_out_dev=None), dict(k_out_dev=None), dict(pos_dev=None),
               dict(turns_dev=None), dict(q_dev=OK + 1), dict(k_out_dev=OK + 1),
               dict(k_dev=ODD, dtype=B.HS_DTYPE_FP32), dict(q_weight_dev=ODD),
               dict(k_weight_dev=ODD), dict(pos_dev=ODD), dict(turns_dev=OK + 4),
               dict(axis_dev=ODD), dict(count_dev=ODD)):
        assert call(**kw) == bad, kw
    for kw in (dict(head_dim=80), dict(head_dim=512, rot_dim=0), dict(num_axes=5),
               dict(batch=1 << 20, tokens=1 << 10), dict(num_heads=1 << 21)):
        assert call(**kw) == unsupported, kw
    for kw in (dict(batch=0), dict(tokens=0), dict(num_heads=0, num_kv_heads=0)):
        assert call(q_dev=None, k_dev=None, **kw) == B.HS_OK, kw


def test_bound_keys_refuses(lib):
    base = dict(k=OK, stride=STRIDES, dtype=B.HS_DTYPE_BF16, heads=2, dim=64, T=16, req=OK,
                start=OK, count=OK, batch=1, m=4, bounds=OK, R=1, L=64)

    def call(**kw):
        a = dict(base, **kw)
        return lib.hs_bound_keys(a["k"], a["stride"], a["dtype"], a["heads"], a["dim"], a["T"],
                                 a["req"], a["start"], a["count"], a["batch"], a["m"],
                                 a["bounds"], a["R"], a["L"], None)

    for kw in (dict(stride=None), dict(batch=-1), dict(m=-1), dict(R=0), dict(L=0),
               dict(heads=0), dict(dim=0), dict(T=0), dict(dtype=B.HS_DTYPE_FP32), dict(dtype=-1),
               dict(k=None), dict(req=None), dict(start=None), dict(count=None),
               dict(bounds=None), dict(k=OK + 1), dict(bounds=OK + 1), dict(req=ODD),
               dict(start=ODD), dict(count=ODD)):
        assert call(**kw) == bad, kw
    for kw in (dict(dim=80), dict(heads=129), dict(T=4097), dict(batch=1 << 20, m=1 << 20, T=1)):
        assert call(**kw) == unsupported, kw
    assert call(batch=0) == B.HS_OK and call(m=0) == B.HS_OK


def _select(lib, **kw):
    base = dict(q_dev=OK, bounds_dev=OK, dtype=B.HS_DTYPE_BF16, batch=2, steps=2, num_heads=8,
                num_kv_heads=2, head_dim=64, num_requests=4, max_seq_len=1000, block_tokens=16,
                select=8, first=1, last=2, q_stride=STRIDES, req_dev=OK, seq_lens_dev=OK,
                blocks_dev=OK, topk_dev=OK, scores_dev=OK, workspace_dev=OK,
                workspace_bytes=1 << 20)
    return lib.hs_select_blocks(ctypes.byref(B._HsSelectArgs(**dict(base, **kw))), None)


def test_select_blocks_refuses(lib):
    assert lib.hs_select_blocks(None, None) == bad
    for kw in (dict(batch=-1), dict(steps=0), dict(num_heads=0), dict(num_kv_heads=0),
               dict(num_heads=7), dict(head_dim=0), dict(num_requests=0), dict(max_seq_len=0),
               dict(block_tokens=0), dict(select=0), dict(first=-1), dict(last=-1), dict(first=9),
               dict(first=6, last=3), dict(first=2 ** 31 - 1, last=2 ** 31 - 1),
               dict(dtype=B.HS_DTYPE_FP32), dict(dtype=-1), dict(q_dev=None),
               dict(bounds_dev=None), dict(req_dev=None), dict(seq_lens_dev=None),
               dict(topk_dev=None), dict(scores_dev=None), dict(workspace_dev=None),
               dict(q_dev=OK + 1), dict(bounds_dev=OK + 1), dict(req_dev=ODD),
               dict(seq_lens_dev=ODD), dict(blocks_dev=ODD), dict(topk_dev=ODD),
               dict(scores_dev=ODD), dict(workspace_dev=ODD), dict(workspace_bytes=8)):
        assert _select(lib, **kw) == bad, kw
    for kw in (dict(steps=5), dict(head_dim=80), dict(block_tokens=5000),
               dict(max_seq_len=16385 * 16), dict(num_heads=256, num_kv_heads=2),
               dict(num_heads=256, num_kv_heads=256), dict(num_heads=64, num_kv_heads=64,
                                                           head_dim=192),
               dict(num_heads=64, num_kv_heads=64, head_dim=128, steps=3), dict(select=16385),
               dict(batch=1 << 30)):
        assert _select(lib, **kw) == unsupported, kw
    assert _select(lib, batch=0, q_dev=None) == B.HS_OK
    n = pkg.hs_select_workspace_bytes(2, 2, 1000, 16)
    assert n == 4 * 2 * 2 * 8 and pkg.hs_select_workspace_bytes(0, 1, 1, 1) == 0
    for sizes in ((-1, 1, 1, 1), (1, 0, 1, 1), (1, 5, 1, 1), (1, 1, 0, 1), (1, 1, 1, 0),
                  (1, 1, 16385, 1)):
        with pytest.raises(pkg.HsError):
            pkg.hs_select_workspace_bytes(*sizes)


def test_attend_prefix_refuses(lib):
    fmt = pkg.make_kv_format(2, 64, 16)
    base = dict(q_dev=OK, out_dev=OK, dtype=B.HS_DTYPE_BF16, batch=2, steps=2, num_heads=8,
                num_requests=3, max_seq_len=100, num_prefixes=2, sm_scale=0.1, q_stride=STRIDES,
                out_stride=STRIDES, join_stride=STRIDES, rows_dev=OK, scales_dev=OK,
                prefix_dev=OK, lens_dev=OK, starts_dev=OK, lse_dev=OK, join_out_dev=OK,
                join_lse_dev=OK, workspace_dev=OK, workspace_bytes=1 << 40)

    def call(f=fmt, **kw):
        args = B._HsPrefixArgs(**dict(base, **kw))
        return lib.hs_attend_prefix(ctypes.byref(f), ctypes.byref(args), None)

    assert lib.hs_attend_prefix(ctypes.byref(fmt), None, None) == bad
    assert lib.hs_attend_prefix(None, ctypes.byref(B._HsPrefixArgs(**base)), None) == bad
    assert call(f=B.HsKvFormat(2, 100, 16, 0, 400)) == unsupported
    for kw in (dict(batch=-1), dict(steps=0), dict(num_heads=0), dict(num_heads=7),
               dict(num_requests=0), dict(max_seq_len=0), dict(num_prefixes=-1),
               dict(dtype=B.HS_DTYPE_FP32), dict(dtype=-1), dict(q_dev=None), dict(out_dev=None),
               dict(rows_dev=None), dict(scales_dev=None), dict(prefix_dev=None),
               dict(lens_dev=None), dict(starts_dev=None), dict(join_out_dev=None),
               dict(join_lse_dev=None), dict(workspace_dev=None), dict(q_dev=OK + 1),
               dict(out_dev=OK + 1), dict(join_out_dev=OK + 1), dict(rows_dev=OK + 8),
               dict(scales_dev=ODD), dict(prefix_dev=ODD), dict(lens_dev=ODD),
               dict(starts_dev=ODD), dict(lse_dev=ODD), dict(join_lse_dev=ODD),
               dict(workspace_dev=OK + 8), dict(workspace_bytes=64)):
        assert call(**kw) == bad, kw
    for kw in (dict(num_heads=130), dict(num_prefixes=257), dict(batch=1 << 30)):
        assert call(**kw) == unsupported, kw
    # tiles: 2 heads, (batch * 8 rows of a head / 128 + 2) by (max_seq_len / 64)
    for kw in (dict(batch=1 << 17, steps=2, max_seq_len=2 ** 31 - 1),
               dict(batch=1 << 24, steps=2, max_seq_len=1 << 16)):
        assert call(**kw) == unsupported, kw
    wide = pkg.make_kv_format(2, 64, 16, item_size_bytes=1024)
    assert call(f=wide, max_seq_len=1 << 30) == unsupported
    assert call(batch=0, q_dev=None) == B.HS_OK
    assert pkg.hs_prefix_workspace_bytes(fmt, 0, 1, 8, 1) == 0
    assert pkg.hs_prefix_workspace_bytes(fmt, 4, 1, 8, 1) > 0
    with pytest.raises(pkg.HsError):
        pkg.hs_prefix_workspace_bytes(fmt, 4, 1, 7, 1)


def test_make_rope():
    freq = ref.frequencies(64)
    r = pkg.make_rope(freq, device="cpu")
    assert r.rot_dim == 64 and r.num_axes == 1 and r.axis is None and not r.adjacent
    for f, t in zip(freq, r.turns.tolist()):  # parts of a turn
        assert abs((t % 2 ** 64) / 2 ** 64 - f / (2 * math.pi)) < 2.0 ** -53
    r = pkg.make_rope(torch.tensor([2 * math.pi * x for x in (0.25, 1.75, -0.25, 0)] * 2,
                                   dtype=torch.float64), [0, 2, 1, 0] * 2, True, "cpu")
    assert r.num_axes == 3 and r.adjacent and r.axis.tolist() == [0, 2, 1, 0] * 2
    assert r.turns.tolist() == [2 ** 62, -2 ** 62, -2 ** 62, 0] * 2
    assert pkg.make_rope([], device="cpu").rot_dim == 0
    for args in (([1.0] * 7,), ([math.inf] * 8,), ([1.0] * 8, [0] * 7), ([1.0] * 8, [4] * 8),
                 ([1.0] * 8, [-1] * 8)):
        with pytest.raises(ValueError):
            pkg.make_rope(*args, device="cpu")


def test_binding_refuses_shapes(lib):
    """Shapes and types are checked before addresses."""
    bf = torch.bfloat16
    q, k = torch.zeros((2, 3, 8, 64), dtype=bf), torch.zeros((2, 3, 2, 64), dtype=bf)
    one = torch.zeros(2, dtype=torch.int32)
    rope = pkg.make_rope(ref.frequencies(64), device="cpu")
    pos = torch.zeros((1, 2, 3), dtype=torch.int32)

    def rotate(q=q, k=k, pos=pos, q_out=q, k_out=k, **kw):
        pkg.hs_norm_rope(q, k, pos, rope, q_out, k_out, **kw)

    for kw in (dict(q=None), dict(q_out=None), dict(q=None, k=None, q_out=None, k_out=None),
               dict(q=q[0]), dict(k=k[:1]), dict(k=k[..., :32]), dict(q_out=q[:, :2]),
               dict(k=k.half()), dict(k_out=k.half()), dict(pos=pos[:, :1]), dict(pos=None),
               dict(pos=pos.expand(2, 2, 3)), dict(q_weight=torch.zeros(32)),
               dict(count=one[:1]), dict()):
        with pytest.raises(ValueError):
            rotate(**kw)

    bounds = torch.zeros((4, 5, 2, 2, 64), dtype=bf)
    assert pkg.bounds_shape(4, 70, 16, 2, 64) == bounds.shape

    def bound(k=k, req=one, start=one, count=one, T=16, L=70, bounds=bounds):
        pkg.hs_bound_keys(k, req, start, count, T, L, bounds)

    for kw in (dict(k=k[0]), dict(req=one[:1]), dict(start=one[:1]), dict(count=one[:1]),
               dict(T=8), dict(T=0), dict(L=0), dict(L=100), dict(bounds=bounds[:, :4]),
               dict(bounds=bounds.half()), dict(k=k.float(), bounds=bounds.float()), dict()):
        with pytest.raises(ValueError):
            bound(**kw)

    topk = torch.zeros((2, 3, 48), dtype=torch.int32)
    blocks, scores = torch.zeros((2, 3, 3), dtype=torch.int32), torch.zeros((2, 3, 5))
    ws = torch.zeros(64, dtype=torch.uint8)

    def select(q=q, bounds=bounds, req=one, lens=one, T=16, L=70, blocks=blocks, topk=topk,
               scores=scores):
        pkg.hs_select_blocks(q, bounds, req, lens, T, L, 1, 1, blocks, topk, scores, ws)

    for kw in (dict(q=q[0]), dict(q=q.half()), dict(bounds=bounds[0]), dict(bounds=bounds[:, 1:]),
               dict(req=one[:1]), dict(lens=one[:1]), dict(T=0), dict(T=15),
               dict(topk=topk[:, :, :40]), dict(topk=topk[:1]), dict(blocks=blocks[..., :2]),
               dict(scores=scores[..., :4]), dict()):
        with pytest.raises(ValueError):
            select(**kw)

    fmt = pkg.make_kv_format(2, 64, 16)
    rows, scales = torch.zeros((4, 70, 256), dtype=torch.uint8), torch.zeros((4, 5, 2, 2))
    starts, lse = torch.zeros(3, dtype=torch.int32), torch.zeros((2, 3, 8))

    def prefix(q=q, rows=rows, scales=scales, prefix=one, lens=one, starts=starts, out=q, lse=lse,
               **kw):
        pkg.hs_attend_prefix(fmt, q, rows, scales, prefix, lens, starts, out, lse=lse, **kw)

    for kw in (dict(q=q[0]), dict(q=q[..., :32]), dict(rows=rows[..., :128]), dict(rows=rows[0]),
               dict(scales=scales[:, :4]), dict(prefix=one[:1]), dict(lens=one[:1]),
               dict(starts=starts[:2]), dict(out=q[:1]), dict(out=q.half()), dict(lse=lse[:1]),
               dict(join_out=q), dict(join_lse=lse), dict(join_out=q.half(), join_lse=lse),
               dict(join_out=q[:, :, :4], join_lse=lse), dict(join_out=q, join_lse=lse[:1]), dict()):
        with pytest.raises(ValueError):
            prefix(**kw)


def test_cache_refuses():
    from sparse_attention_kv_swap_gb300.cache import SwapInCache
    cache = SwapInCache.__new__(SwapInCache)  # the sizes alone are looked at
    cache.cfg, cache.device = pkg.make_config(4, 70, 256, 48, 48, 1), torch.device("cpu")
    fmt = pkg.make_kv_format(2, 64, 16)
    bounds = cache.key_bounds(fmt, torch.bfloat16, 16)
    assert bounds.shape == (4, 5, 2, 2, 64) and bounds.dtype is torch.bfloat16
    q, one = torch.zeros((2, 3, 8, 64), dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    for T in (0, -1, 32, 96):
        with pytest.raises(ValueError):
            cache.select_blocks(bounds, T, q, one, one)
    with pytest.raises(ValueError):
        cache.select_blocks(bounds[:, 1:], 16, q, one, one)
    with pytest.raises(ValueError):
        cache.bound_keys(bounds, 16, q, one, one, one)


# ---- the plain implementation itself ---------------------------------------------------

def test_reference_bounds_are_bounds():
    """A block's score is no less than the sum over the query heads of q . k for its tokens."""
    rng = np.random.default_rng(0)
    k, q = rng.standard_normal((1, 50, 2, 32)), rng.standard_normal((1, 1, 6, 32))
    bounds = np.zeros((1, 4, 2, 2, 32))
    ref.bound(k, [0], [0], [50], 16, 64, bounds)
    z, _ = ref.scores(q, bounds, [0], [50], 16, 64)
    for t in range(50):
        dot = (q[0, 0].reshape(2, 3, 32) * k[0, t][:, None]).sum()
        assert z[0, 0, t // 16] >= dot
    blocks, topk = ref.select(z, [50], [0], 1, 16, 64, 2, 0, 1)
    assert blocks[0, 0, 1] == 3 and topk[0, 0, -1] == -1 and topk[0, 0, 17] == 49


def test_reference_join_of_parts_is_the_whole():
    rng = np.random.default_rng(1)
    q = rng.standard_normal((2, 1, 4, 32))
    rows = rng.integers(0, 120, (1, 40, 128)).astype(np.uint8)
    scales = np.full((1, 40, 2, 2), 2.0 ** -6, np.float32)
    args = ([0], [0, 2], 1, 2, "int8", 0.1)

    def over(r, n, join=None):
        return ref.attend(q, r, scales, args[0], [n], *args[1:], join=join)

    whole, first = over(rows, 40), over(rows, 25)
    both = over(rows[:, 25:], 15, (first["out"], first["lse"]))
    assert np.allclose(both["out"], whole["out"]) and np.allclose(both["lse"], whole["lse"])
