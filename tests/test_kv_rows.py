"""The 8-bit key/value row calls on the CPU: what they refuse, before any
launch, at the C entry points and in the Python binding, and the layout of the
structures that cross it."""
import ctypes
import re

import numpy as np
import pytest
import torch

import kv_reference as ref
import sparse_attention_kv_swap_gb300 as pkg
from sparse_attention_kv_swap_gb300 import binding as B


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_kv_swap_gb300 import build
    build.build()
    return B.load_library()


def _fmt(**kw):
    base = dict(num_kv_heads=8, head_dim=128, block_tokens=64, code=B.HS_KV_E4M3,
                item_size_bytes=2048)
    base.update(kw)
    return B.HsKvFormat(**base)


def _check(lib, **kw):
    return lib.hs_kv_format_check(ctypes.byref(_fmt(**kw)))


def test_header_constants_and_structs(lib):
    text = open(B.HEADER).read()
    consts = dict(re.findall(r"#define (HS_(?:KV|DTYPE|MAX_KV)_[A-Z0-9_]+) (\d+)", text))
    for name in ("HS_KV_E4M3", "HS_KV_INT8", "HS_DTYPE_BF16", "HS_DTYPE_FP16", "HS_DTYPE_FP32",
                 "HS_MAX_KV_BLOCK", "HS_MAX_KV_HEADS"):
        assert int(consts[name]) == getattr(B, name), name
    code = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    for struct, cls in (("hs_kv_format", B.HsKvFormat), ("hs_kv_input", B._HsKvInput),
                        ("hs_attend_args", B._HsAttendArgs)):
        body = re.search(r"typedef struct %s \{(.*?)\}" % struct, code, re.S).group(1)
        names = []
        for decl in body.split(";"):
            decl = decl.strip()
            if decl:
                first = decl.split(",")
                names += [re.findall(r"(\w+)(?:\[\d+\])?$", part.strip())[0] for part in first]
        assert names == [n for n, _ in cls._fields_], struct
    # the packed forms that the binding passes have the same layout
    for cls, pack in ((B._HsAttendArgs, B._ATTEND_ARGS), (B._HsKvInput, B._KV_INPUT)):
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


def test_format_check(lib):
    assert _check(lib) == B.HS_OK
    for dim in (32, 64, 96, 128, 192, 256):
        assert _check(lib, num_kv_heads=1, head_dim=dim) == B.HS_OK
    for dim in (16, 48, 80, 160, 512):
        assert _check(lib, num_kv_heads=1, head_dim=dim) == B.HS_ERR_UNSUPPORTED
    assert _check(lib, head_dim=0) == B.HS_ERR_INVALID_ARG
    assert _check(lib, num_kv_heads=0) == B.HS_ERR_INVALID_ARG
    assert _check(lib, num_kv_heads=129, head_dim=32,
                  item_size_bytes=16384) == B.HS_ERR_UNSUPPORTED
    assert _check(lib, block_tokens=0) == B.HS_ERR_INVALID_ARG
    assert _check(lib, block_tokens=B.HS_MAX_KV_BLOCK + 1) == B.HS_ERR_UNSUPPORTED
    assert _check(lib, code=2) == B.HS_ERR_INVALID_ARG
    assert _check(lib, item_size_bytes=2047) == B.HS_ERR_INVALID_ARG
    assert _check(lib, item_size_bytes=2032) == B.HS_ERR_INVALID_ARG  # too narrow
    assert _check(lib, item_size_bytes=2064) == B.HS_OK  # padded
    assert _check(lib, num_kv_heads=128, head_dim=256,
                  item_size_bytes=65536) == B.HS_OK
    assert _check(lib, item_size_bytes=B.HS_MAX_ITEM_BYTES + 16) == B.HS_ERR_UNSUPPORTED
    assert lib.hs_kv_format_check(None) == B.HS_ERR_INVALID_ARG
    with pytest.raises(pkg.HsError):
        pkg.make_kv_format(8, 100, 64)
    assert pkg.make_kv_format(5, 64, 16, item_size_bytes=656).item_size_bytes == 656


# Addresses below are never dereferenced: every call is refused on the host.
OK, ODD = 0x20000, 0x20002


def _input(**kw):
    z = (ctypes.c_int64 * 3)(1, 1, 1)
    base = dict(k_dev=OK, v_dev=OK, dtype=B.HS_DTYPE_BF16, k_stride=z, v_stride=z)
    base.update(kw)
    return B._HsKvInput(**base)


def test_quantize_refuses(lib):
    f = _fmt()

    def call(fmt=f, inp=None, req=OK, start=OK, count=OK, batch=1, m=1, rows=OK, scales=OK, R=1,
             L=64):
        inp = _input() if inp is None else inp
        return lib.hs_quantize_kv(ctypes.byref(fmt), ctypes.byref(inp), req, start, count, batch,
                                  m, rows, scales, R, L, None)

    bad = B.HS_ERR_INVALID_ARG
    assert call(fmt=_fmt(head_dim=100)) == B.HS_ERR_UNSUPPORTED
    assert lib.hs_quantize_kv(ctypes.byref(f), None, OK, OK, OK, 1, 1, OK, OK, 1, 64, None) == bad
    for kw in (dict(batch=-1), dict(m=-1), dict(R=0), dict(L=0), dict(req=None), dict(start=None),
               dict(count=None), dict(rows=None), dict(scales=None), dict(req=ODD),
               dict(start=ODD), dict(count=ODD), dict(scales=ODD), dict(rows=OK + 8),
               dict(inp=_input(k_dev=None)), dict(inp=_input(v_dev=None)),
               dict(inp=_input(dtype=3)), dict(inp=_input(dtype=-1)),
               dict(inp=_input(k_dev=OK + 1)),
               dict(inp=_input(v_dev=ODD, dtype=B.HS_DTYPE_FP32))):
        assert call(**kw) == bad, kw
    assert call(batch=1 << 20, m=1 << 20) == B.HS_ERR_UNSUPPORTED
    assert call(batch=0) == B.HS_OK and call(m=0) == B.HS_OK


def test_append_refuses_without_a_handle(lib):
    f, inp = _fmt(), _input()
    assert lib.hs_append_kv(None, 0, ctypes.byref(f), ctypes.byref(inp), OK, OK, OK, 1, 1, OK,
                            None) == B.HS_ERR_INVALID_ARG


def _attend_args(**kw):
    z = (ctypes.c_int64 * 3)(1, 1, 1)
    base = dict(q_dev=OK, out_dev=OK, dtype=B.HS_DTYPE_BF16, batch=1, steps=1, top_k=16,
                num_heads=8, num_requests=1, max_seq_len=64, sm_scale=1.0, q_stride=z,
                out_stride=z, rows_dev=OK, num_rows=16, locs_dev=OK, topk_dev=OK, req_dev=OK,
                scales_dev=OK, lse_dev=None, weights_dev=None, acc_dev=None, workspace_dev=None,
                workspace_bytes=0)
    base.update(kw)
    return B._HsAttendArgs(**base)


def test_attend_refuses(lib):
    f = _fmt()

    def call(fmt=f, **kw):
        a = _attend_args(**kw)
        return lib.hs_attend(ctypes.byref(fmt), ctypes.byref(a), None)

    bad = B.HS_ERR_INVALID_ARG
    assert lib.hs_attend(ctypes.byref(f), None, None) == bad
    assert call(fmt=_fmt(head_dim=100)) == B.HS_ERR_UNSUPPORTED
    for kw in (dict(batch=-1), dict(steps=0), dict(top_k=-1), dict(num_heads=0),
               dict(num_heads=12), dict(num_requests=0), dict(max_seq_len=0), dict(num_rows=-1),
               dict(dtype=B.HS_DTYPE_FP32), dict(dtype=-1), dict(q_dev=None), dict(out_dev=None),
               dict(req_dev=None), dict(locs_dev=None), dict(topk_dev=None),
               dict(scales_dev=None), dict(rows_dev=None), dict(q_dev=OK + 1),
               dict(out_dev=OK + 1), dict(rows_dev=OK + 8), dict(locs_dev=ODD),
               dict(topk_dev=ODD), dict(req_dev=ODD), dict(scales_dev=ODD), dict(lse_dev=ODD),
               dict(weights_dev=ODD), dict(acc_dev=ODD), dict(workspace_dev=OK + 8),
               dict(steps=2, acc_dev=OK)):
        assert call(**kw) == bad, kw
    assert call(num_heads=136) == B.HS_ERR_UNSUPPORTED
    assert call(top_k=(1 << 22) + 1) == B.HS_ERR_UNSUPPORTED
    assert call(batch=0) == B.HS_OK


def test_attend_workspace(lib):
    """Only sizes whose scores do not fit the shared memory of 16 CTAs need a workspace,
    and a call without enough of it is refused."""
    f = pkg.make_kv_format(8, 128, 64)
    assert pkg.hs_attend_workspace_bytes(f, 64, 4, 2048, 64) == 0
    assert pkg.hs_attend_workspace_bytes(f, 16, 1, 8192, 64) == 0
    assert pkg.hs_attend_workspace_bytes(f, 0, 1, 1 << 20, 64) == 0
    need = pkg.hs_attend_workspace_bytes(f, 2, 3, 40000, 64)
    # scores, scales, locations and positions of every entry
    assert need >= 2 * 3 * 40000 * 4 * (64 + 16 + 2)
    assert need <= 2 * 3 * 40000 * 4 * (64 + 16 + 2) * 1.1
    with pytest.raises(pkg.HsError):
        pkg.hs_attend_workspace_bytes(f, 1, 0, 64, 64)
    for ws, n in ((None, need), (OK, need - 1)):
        a = _attend_args(batch=2, steps=3, top_k=40000, num_heads=64, workspace_dev=ws,
                         workspace_bytes=n)
        assert lib.hs_attend(ctypes.byref(f), ctypes.byref(a), None) == B.HS_ERR_INVALID_ARG


def test_accumulate_and_evict_refuse(lib):
    bad = B.HS_ERR_INVALID_ARG

    def acc(w=OK, t=OK, r=OK, n=None, b=1, s=1, k=4, a=OK, R=1, L=8):
        return lib.hs_accumulate(w, t, r, n, b, s, k, a, R, L, None)

    for kw in (dict(b=-1), dict(s=0), dict(k=-1), dict(R=0), dict(L=0), dict(w=None),
               dict(t=None), dict(r=None), dict(a=None), dict(w=ODD), dict(t=ODD), dict(r=ODD),
               dict(n=ODD), dict(a=ODD)):
        assert acc(**kw) == bad, kw
    assert acc(b=0) == B.HS_OK and acc(k=0) == B.HS_OK

    def ev(a=OK, r=OK, n=OK, b=1, recent=1, budget=4, R=1, L=8, keep=OK, kept=OK, ka=OK):
        return lib.hs_evict(a, r, n, b, recent, budget, R, L, keep, kept, ka, None)

    for kw in (dict(b=-1), dict(recent=-1), dict(recent=5), dict(budget=0, recent=0), dict(R=0),
               dict(L=0), dict(a=None), dict(r=None), dict(n=None), dict(keep=None),
               dict(kept=None), dict(a=ODD), dict(r=ODD), dict(n=ODD), dict(keep=ODD),
               dict(kept=ODD), dict(ka=ODD)):
        assert ev(**kw) == bad, kw
    assert ev(L=(1 << 30) + 1) == B.HS_ERR_UNSUPPORTED
    assert ev(b=0) == B.HS_OK


def test_compact_refuses(lib):
    f = _fmt()
    src, dst = 0x1000000, 0x2000000

    def call(fmt=f, s=src, ss=OK, sR=2, sL=64, sq=OK, keep=OK, kept=OK, b=1, budget=32, d=dst,
             ds=OK, dR=2, dL=64, dq=OK):
        return lib.hs_compact_kv(ctypes.byref(fmt), s, ss, sR, sL, sq, keep, kept, b, budget, d,
                                 ds, dR, dL, dq, None)

    bad = B.HS_ERR_INVALID_ARG
    assert call(fmt=_fmt(head_dim=100)) == B.HS_ERR_UNSUPPORTED
    for kw in (dict(b=-1), dict(budget=0), dict(sR=0), dict(sL=0), dict(dR=0), dict(dL=0),
               dict(s=None), dict(ss=None), dict(sq=None), dict(keep=None), dict(kept=None),
               dict(d=None), dict(ds=None), dict(dq=None), dict(s=src + 8), dict(d=dst + 8),
               dict(ss=ODD), dict(ds=ODD), dict(sq=ODD), dict(dq=ODD), dict(keep=ODD),
               dict(kept=ODD), dict(d=src), dict(d=src + 2 * 64 * 2048 - 16),
               dict(s=dst + 2 * 64 * 2048 - 16)):
        assert call(**kw) == bad, kw
    assert call(b=0) == B.HS_OK


def test_binding_checks_shapes_and_memory(lib):
    """Shapes, dtypes and memory kinds are refused before the library is called."""
    fmt = pkg.make_kv_format(2, 64, 16)
    i32, f32 = dict(dtype=torch.int32), dict(dtype=torch.float32)
    kv = torch.zeros((3, 4, 2, 64), dtype=torch.bfloat16)
    one = torch.zeros(3, **i32)
    rows = torch.zeros((5, 40, 256), dtype=torch.uint8)
    scales = torch.zeros((5, 3, 2, 2), **f32)
    with pytest.raises(ValueError, match="rows"):
        pkg.hs_quantize_kv(fmt, kv, kv, one, one, one, rows[..., :128], scales)
    with pytest.raises(ValueError, match="scales"):
        pkg.hs_quantize_kv(fmt, kv, kv, one, one, one, rows, scales[:, :2])
    with pytest.raises(ValueError, match="k must be"):
        pkg.hs_quantize_kv(fmt, kv[..., :32], kv, one, one, one, rows, scales)
    with pytest.raises(ValueError, match="v must"):
        pkg.hs_quantize_kv(fmt, kv, kv[:, :3], one, one, one, rows, scales)
    with pytest.raises(ValueError, match="dtype"):
        pkg.hs_quantize_kv(fmt, kv, kv.half(), one, one, one, rows, scales)
    with pytest.raises(ValueError, match="count"):
        pkg.hs_quantize_kv(fmt, kv, kv, one, one, one[:2], rows, scales)
    with pytest.raises(ValueError, match="device memory"):
        pkg.hs_quantize_kv(fmt, kv, kv, one, one, one, rows, scales)

    q = torch.zeros((3, 2, 8, 64), dtype=torch.float16)
    locs = torch.zeros((3, 2, 16), **i32)

    def attend(q=q, locs=locs, topk=locs, req=one, scales=scales, L=40, out=q, **kw):
        pkg.hs_attend(fmt, q, rows, locs, topk, req, scales, L, out, **kw)

    for match, kw in (("q must", dict(q=q[..., :32])), ("topk", dict(topk=locs[:2])),
                      ("out must have q's", dict(out=q.float())), ("out", dict(out=q[:2])),
                      ("locs", dict(locs=locs[:, :, :3])), ("req", dict(req=one[:2])),
                      ("scales", dict(scales=scales[:, :2])),
                      ("lse", dict(lse=torch.zeros((3, 2, 4), **f32))),
                      ("weights", dict(weights=torch.zeros((3, 2, 4), **f32))),
                      ("acc", dict(acc=torch.zeros((5, 41), **f32))),
                      ("device memory", dict())):
        with pytest.raises(ValueError, match=match):
            attend(**kw)
    with pytest.raises(ValueError, match="weights"):
        pkg.hs_accumulate(torch.zeros((3, 2, 4)), locs, one, torch.zeros((5, 40)))
    with pytest.raises(ValueError, match="keep"):
        pkg.hs_evict(torch.zeros((5, 40)), one, one, 1, one, one)
    with pytest.raises(ValueError, match="kept"):
        pkg.hs_evict(torch.zeros((5, 40)), one, one, 1, torch.zeros((3, 8), **i32), one[:2])
    with pytest.raises(ValueError, match="dst_scales"):
        pkg.hs_compact_kv(fmt, rows, scales, one, torch.zeros((3, 8), **i32), one, rows,
                          scales[:4], one)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_reference_codes(code):
    """The plain implementation's own codes: every finite code survives a round trip under
    its scale, and a value is off by half a step at most."""
    table = ref.decode_table(code)
    x = torch.tensor(table[np.isfinite(table)], dtype=torch.float32)
    x = x[x.abs() <= (448 if code == "e4m3" else 127)]
    s = ref.scale_of(x.abs().max(), code)
    assert float(s) == 1.0
    back = ref.encode(x, s.expand_as(x), code)
    assert np.array_equal(table[back.numpy()], x.numpy().astype(np.float64))
    g = torch.Generator().manual_seed(3)
    y = torch.randn(4000, generator=g) * torch.exp(4 * torch.randn(4000, generator=g))
    s = ref.scale_of(y.abs().max(), code)
    z = table[ref.encode(y, s.expand_as(y), code).numpy()] * float(s)
    step = (np.maximum(np.abs(y.numpy()) * 2.0 ** -4, float(s) * 2.0 ** -10) if code == "e4m3"
            else float(s) * 0.5 * (1 + 2.0 ** -15))
    assert (np.abs(z - y.numpy().astype(np.float64)) <= step).all()


def test_reference_eviction_is_a_stable_sort():
    rng = np.random.default_rng(5)
    acc = rng.integers(0, 6, size=(2, 50)).astype(np.float32)
    acc[1, 7] = np.nan
    keep, kept, kept_acc = ref.evict(acc, [1, 0], [50, 9], 5, 20)
    assert kept.tolist() == [20, 9] and (keep[0, -5:] == np.arange(45, 50)).all()
    assert (np.diff(keep[0]) > 0).all() and 7 not in keep[0]
    low = acc[1, keep[0, :15]].min()
    out = np.setdiff1d(np.arange(45), keep[0])
    assert (np.nan_to_num(acc[1, out], nan=-1) <= low).all()
    ties = np.nonzero(acc[1, :45] == low)[0]
    n = (acc[1, keep[0, :15]] == low).sum()
    assert (keep[0, :15][acc[1, keep[0, :15]] == low] == ties[:n]).all()
