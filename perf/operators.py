"""Cases of the 8-bit cache operators: attention over block-scaled rows at
device locations, quantisation of new keys and values into such rows, and
eviction by accumulated attention weight with the compaction it asks for.

A cache row of W bytes holds one token: the K codes of every head, then the V
codes.  scales[q, t // T, c, h] is the scale of K (c = 0) or V (c = 1) of the
T tokens of that block of request q.  ``own`` selects the framework's calls;
otherwise the same results come from elementary torch operations in 32 bits.
"""
import functools
import math

import torch

own = False

E4M3_MAX, INT8_MAX = 448.0, 127.0
SCALE_FLOOR = 2.0 ** -100  # smallest magnitude the scales are made for


# ---- the cases ----------------------------------------------------------------

def _attend(name, B, S, K, L, slots, heads, group, dim, block, dtype, code, holes):
    return dict(name=name, op="attend", B=B, S=S, K=K, L=L, slots=slots, heads=heads, group=group,
                dim=dim, block=block, dtype=dtype, code=code, holes=holes)


def _quantize(name, B, M, L, heads, dim, block, dtype, code, ragged):
    return dict(name=name, op="quantize", B=B, M=M, L=L, heads=heads, dim=dim, block=block,
                dtype=dtype, code=code, ragged=ragged)


def _evict(name, B, L, budget, recent, heads, dim, block, code, ragged):
    return dict(name=name, op="evict", B=B, L=L, budget=budget, recent=recent, heads=heads,
                dim=dim, block=block, code=code, ragged=ragged)


def listed():
    return [
        # One request, 64 selected tokens: the smallest decode step (single-step selection
        # over a 4096-token sequence); only latency counts.
        _attend("attend_one_request", 1, 1, 64, 4096, 320, 2, 4, 128, 16, "bf16", "e4m3", False),
        # A full single-step decode batch: 64 requests, 2048 selected of 32768 tokens, each
        # with a hot buffer of 4096 slots and its scratch rows.
        _attend("attend_decode_batch", 64, 1, 2048, 32768, 6144, 8, 8, 128, 64, "bf16", "e4m3",
                False),
        # Multi-token prediction: 4 steps whose selections overlap by 70 per cent.
        _attend("attend_four_steps", 64, 4, 2048, 32768, 16384, 4, 8, 128, 64, "bf16", "e4m3",
                False),
        # A small serving batch of odd sizes, int8 codes, short requests with empty places.
        _attend("attend_odd_int8", 7, 3, 777, 9973, 2500, 5, 3, 96, 48, "fp16", "int8", True),
        # One shared key/value head (multi-query), 4 steps over a 65536-token context.
        _attend("attend_shared_head", 8, 4, 2048, 65536, 10240, 1, 16, 256, 32, "fp16", "e4m3",
                False),
        # Long context: 8192 selected tokens of 131072, pages of 256 tokens.
        _attend("attend_long_context", 16, 1, 8192, 131072, 16384, 8, 4, 64, 256, "bf16", "e4m3",
                True),
        # One decoded token for each of 64 requests, into blocks that are still filling.
        _quantize("quantize_token", 64, 1, 512, 8, 128, 64, "bf16", "e4m3", True),
        # Prompts of 8192 tokens: whole blocks, bandwidth counts.
        _quantize("quantize_prompt", 4, 8192, 8192, 8, 128, 64, "bf16", "e4m3", False),
        # Chunks of a prompt of different lengths, starting inside a block; int8 codes.
        _quantize("quantize_chunks_int8", 6, 1000, 2048, 5, 96, 48, "fp16", "int8", True),
        # One short sequence that has passed its budget.
        _evict("evict_one_request", 1, 1000, 512, 64, 2, 128, 16, "e4m3", False),
        # A batch cut from 4096 tokens to 2048.
        _evict("evict_batch", 64, 4096, 2048, 256, 8, 128, 64, "e4m3", True),
        # A few very long sequences cut to an eighth, int8 codes: selection counts too.
        _evict("evict_long_int8", 8, 131072, 16384, 1024, 1, 128, 64, "int8", True),
    ]


def _spread(rng, low, high):
    """A whole number from low to high, spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "quantize", "evict"])
    dim = rng.choice([64, 96, 128, 128, 192, 256])
    code = rng.choice(["e4m3", "e4m3", "int8"])
    dtype = rng.choice(["bf16", "fp16"])
    heads = rng.choice([1, 2, 3, 4, 5, 8, 8, 12])
    while 2 * heads * dim > 2048:
        heads = rng.choice([1, 2, 3, 4, 5, 8])
    block = rng.choice([16, 32, 48, 64, 128, 256])
    width = 2 * heads * dim
    if op == "attend":
        S = rng.choice([1, 1, 2, 3, 4])
        K = _spread(rng, 1, 8192 // S)
        most = max(1, min(64, 64 * 4 * 2048 * 1024 // (S * K * width)))
        B = _spread(rng, 1, most)
        L = _spread(rng, max(64, 4 * K), 131072)
        group = rng.choice([1, 2, 3, 4, 6, 8, 8, 12, 16])
        while heads * group > 64:
            group = rng.choice([1, 2, 3, 4, 6, 8])
        slots = _union(S, K) + _spread(rng, 1, 4096)
        c = _attend("", B, S, K, L, slots, heads, group, dim, block, dtype, code,
                    rng.random() < 0.3)
    elif op == "quantize":
        M = _spread(rng, 1, 8192)
        B = _spread(rng, 1, max(1, min(64, 4 * 8192 * 2048 // (M * width))))
        c = _quantize("", B, M, M + rng.randrange(1, 512), heads, dim, block, dtype, code,
                      rng.random() < 0.6)
    else:
        L = _spread(rng, 64, 131072)
        B = _spread(rng, 1, max(1, min(64, 64 * 4096 * 2048 // (L * width))))
        budget = max(1, min(L - 1, int(L * rng.uniform(0.1, 0.75))))
        c = _evict("", B, L, budget, rng.randrange(0, budget // 2 + 1), heads, dim, block, code,
                   rng.random() < 0.6)
    del c["name"]
    return c


def _union(S, K):
    """Distinct tokens over S steps of K, each step replacing 30 per cent."""
    return K + (S - 1) * max(1, (3 * K) // 10)


# ---- inputs ---------------------------------------------------------------------

def _torch_dtype(name):
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def _codes(shape, code, gen):
    """8-bit codes of normally distributed values, as bytes."""
    x = torch.randn(shape, device="cuda", dtype=torch.float16, generator=gen)
    if code == "e4m3":
        return x.mul_(90.0).clamp_(-440.0, 440.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.mul_(32.0).round_().clamp_(-127.0, 127.0).to(torch.int8).view(torch.uint8)


def _scales(R, L, block, heads, code, gen):
    """Scales with which the codes stand for values of order one; block by block they
    differ by a factor of a few, as blocks of a real sequence do."""
    shape = (R, -(-L // block), 2, heads)
    if code == "e4m3":
        e = torch.randint(-8, -5, shape, device="cuda", generator=gen)
        return torch.ldexp(torch.ones(shape, device="cuda"), e)
    return (torch.rand(shape, device="cuda", generator=gen) * 0.06 + 0.015)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    return {"attend": _prepare_attend, "quantize": _prepare_quantize,
            "evict": _prepare_evict}[case["op"]](case, gen, s)


def _prepare_attend(c, gen, s):
    B, S, K, L, slots = c["B"], c["S"], c["K"], c["L"], c["slots"]
    heads, dim = c["heads"], c["dim"]
    width = 2 * heads * dim
    s["rows"] = _codes((B * slots, width), c["code"], gen)
    s["scales"] = _scales(B, L, c["block"], heads, c["code"], gen)
    s["q"] = torch.randn((B, S, heads * c["group"], dim), device="cuda",
                         generator=gen).to(_torch_dtype(c["dtype"]))
    s["req"] = torch.randperm(B, device="cuda", generator=gen).to(torch.int32)
    # The call's distinct tokens and the device rows that hold them; each step takes K of them,
    # 70 per cent in common with the step before, in the indexer's (arbitrary) order.
    union = _union(S, K)
    toks = torch.rand((B, L), device="cuda", generator=gen).argsort(dim=1)[:, :union]
    rows = torch.rand((B, slots), device="cuda", generator=gen).argsort(dim=1)[:, :union]
    rows = rows + s["req"].long()[:, None] * slots
    move = max(1, (3 * K) // 10)
    pick = torch.rand((B, S, K), device="cuda", generator=gen).argsort(dim=2)
    pick = pick + torch.arange(S, device="cuda")[None, :, None] * move
    at = pick.reshape(B, S * K)
    topk = toks.gather(1, at).reshape(B, S, K)
    locs = rows.gather(1, at).reshape(B, S, K)
    if c["holes"]:  # requests shorter than the selection leave invalid entries
        part = torch.rand((B, 1, 1), device="cuda", generator=gen) * 0.9 + 0.1
        gone = torch.rand((B, S, K), device="cuda", generator=gen) > part
        topk, locs = topk.masked_fill(gone, -1), locs.masked_fill(gone, -1)
    s["topk"], s["locs"] = topk.to(torch.int32), locs.to(torch.int32)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((B, S, heads * c["group"]), device="cuda")
    s["weights"] = torch.empty((B, S, K), device="cuda")
    s["acc"] = torch.zeros((B, L), device="cuda")
    return s


def _prepare_quantize(c, gen, s):
    B, M, L, heads, dim, T = c["B"], c["M"], c["L"], c["heads"], c["dim"], c["block"]
    # channels differ in size, as those of keys do
    size = torch.exp(0.5 * torch.randn((2, 1, 1, heads, dim), device="cuda", generator=gen))
    for i, name in enumerate(("k", "v")):
        x = torch.randn((B, M, heads, dim), device="cuda", generator=gen) * size[i]
        s[name] = x.to(_torch_dtype(c["dtype"]))
        del x
    s["rows"] = _codes((B, L, 2 * heads * dim), c["code"], gen)
    s["scales"] = _scales(B, L, T, heads, c["code"], gen)
    s["req"] = torch.randperm(B, device="cuda", generator=gen).to(torch.int32)
    if c["ragged"]:
        start = torch.rand(B, device="cuda", generator=gen) * (L - M + 1)
        part = torch.rand(B, device="cuda", generator=gen)
        count = M - (part * (M // 2 + 1)).floor()
    else:
        start = torch.zeros(B, device="cuda")
        count = torch.full((B,), float(M), device="cuda")
    s["start"], s["count"] = start.floor().to(torch.int32), count.to(torch.int32)
    return s


def _prepare_evict(c, gen, s):
    B, L, T, heads, dim = c["B"], c["L"], c["block"], c["heads"], c["dim"]
    width = 2 * heads * dim
    s["rows"] = _codes((B, L, width), c["code"], gen)
    s["scales"] = _scales(B, L, T, heads, c["code"], gen)
    # a few heavy tokens, a long tail of light ones
    s["acc"] = torch.exp(2.5 * torch.randn((B, L), device="cuda", generator=gen))
    s["req"] = torch.randperm(B, device="cuda", generator=gen).to(torch.int32)
    n = torch.full((B,), float(L), device="cuda")
    if c["ragged"]:
        n = L - (torch.rand(B, device="cuda", generator=gen) * (L // 3)).floor()
    s["seq_lens"] = n.to(torch.int32)
    budget, blocks = c["budget"], -(-c["budget"] // T)
    s["keep"] = torch.empty((B, budget), dtype=torch.int32, device="cuda")
    s["kept"] = torch.empty(B, dtype=torch.int32, device="cuda")
    s["kept_acc"] = torch.empty((B, budget), device="cuda")
    s["new_req"] = torch.arange(B, dtype=torch.int32, device="cuda")
    s["new_rows"] = torch.zeros((B, budget, width), dtype=torch.uint8, device="cuda")
    s["new_scales"] = torch.zeros((B, blocks, 2, heads), device="cuda")
    return s


# ---- one pass -------------------------------------------------------------------

@functools.lru_cache(maxsize=None)
def _format(heads, dim, block, code):
    """The cache's row format, which a user's program makes once."""
    import sparse_attention_kv_swap_gb300 as hs
    return hs.make_kv_format(heads, dim, block,
                             hs.HS_KV_E4M3 if code == "e4m3" else hs.HS_KV_INT8)


def run(s):
    op = s["case"]["op"]
    if own:
        return {"attend": _own_attend, "quantize": _own_quantize, "evict": _own_evict}[op](s)
    return {"attend": _plain_attend, "quantize": _plain_quantize, "evict": _plain_evict}[op](s)


def _own_attend(s):
    import sparse_attention_kv_swap_gb300 as hs
    c = s["case"]
    fmt = _format(c["heads"], c["dim"], c["block"], c["code"])
    hs.hs_attend(fmt, s["q"], s["rows"], s["locs"], s["topk"], s["req"], s["scales"], c["L"],
                 s["out"], lse=s["lse"], weights=s["weights"], acc=s["acc"])
    return {"out": s["out"], "lse": s["lse"], "weights": s["weights"], "acc": s["acc"]}


def _own_quantize(s):
    import sparse_attention_kv_swap_gb300 as hs
    c = s["case"]
    fmt = _format(c["heads"], c["dim"], c["block"], c["code"])
    hs.hs_quantize_kv(fmt, s["k"], s["v"], s["req"], s["start"], s["count"], s["rows"],
                      s["scales"])
    return {"codes": s["rows"].view(_code_dtype(c["code"])), "scales": s["scales"]}


def _own_evict(s):
    import sparse_attention_kv_swap_gb300 as hs
    c = s["case"]
    fmt = _format(c["heads"], c["dim"], c["block"], c["code"])
    hs.hs_evict(s["acc"], s["req"], s["seq_lens"], c["recent"], s["keep"], s["kept"],
                s["kept_acc"])
    hs.hs_compact_kv(fmt, s["rows"], s["scales"], s["req"], s["keep"], s["kept"], s["new_rows"],
                     s["new_scales"], s["new_req"])
    return {"keep": s["keep"], "kept": s["kept"], "kept_acc": s["kept_acc"],
            "codes": s["new_rows"].view(_code_dtype(c["code"])), "scales": s["new_scales"]}


def _code_dtype(code):
    return torch.float8_e4m3fn if code == "e4m3" else torch.int8


def _plain_attend(s):
    c = s["case"]
    B, S, K, heads, group, dim = c["B"], c["S"], c["K"], c["heads"], c["group"], c["dim"]
    valid = s["locs"] >= 0
    loc, tok, req = s["locs"].clamp(min=0).long(), s["topk"].clamp(min=0).long(), s["req"].long()
    x = s["rows"][loc].view(_code_dtype(c["code"])).float().view(B, S, K, 2, heads, dim)
    scale = s["scales"][req[:, None, None], tok // c["block"]]  # [B, S, K, 2, heads]
    q = s["q"].float().view(B, S, heads, group, dim)
    # [B, S, heads, group, K]
    logits = torch.matmul(q, x[:, :, :, 0].permute(0, 1, 3, 4, 2))
    logits *= scale[:, :, :, 0].permute(0, 1, 3, 2)[:, :, :, None] * (1.0 / math.sqrt(dim))
    logits = logits.masked_fill(~valid[:, :, None, None], -math.inf)
    top = logits.amax(dim=-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(logits - top)
    total = p.sum(dim=-1, keepdim=True)
    lse = (top + torch.log(total)).reshape(B, S, heads * group)
    p = torch.where(total > 0, p / total, torch.zeros_like(p))
    scaled = p * scale[:, :, :, 1].permute(0, 1, 3, 2)[:, :, :, None]
    out = torch.matmul(scaled, x[:, :, :, 1].permute(0, 1, 3, 2, 4))
    weights = p.sum(dim=(2, 3))
    # what a call adds to a token of an earlier step of the same call comes after that step's
    acc = s["acc"]
    acc.index_put_((req[:, None, None].expand_as(tok), tok),
                   torch.where(valid, weights, torch.zeros_like(weights)), accumulate=True)
    return {"out": out.reshape(B, S, heads * group, dim).to(s["q"].dtype), "lse": lse,
            "weights": weights, "acc": acc}


def _scale_of(peak, code):
    """The scale of blocks whose largest magnitude is `peak` (0 for blocks of zeros)."""
    big = torch.clamp(peak, min=SCALE_FLOOR)
    if code == "e4m3":  # the smallest power of two that brings the peak to 448 or less
        frac, e = torch.frexp(big)
        e = torch.where(frac <= 0.875, e - 9, e - 8)
        s = torch.ldexp(torch.ones_like(big), torch.clamp(e, min=-100))
    else:
        s = big / torch.full_like(big, INT8_MAX)
    return torch.where(peak > 0, s, torch.zeros_like(s))


def _encode(x, scale, code):
    """Codes of x under the scale, which is 0 only where x is."""
    r = torch.where(scale > 0, torch.reciprocal(scale), torch.zeros_like(scale))
    y = x * r
    if code == "e4m3":
        return y.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.round(y).clamp(-INT8_MAX, INT8_MAX).to(torch.int8).view(torch.uint8)


def _plain_quantize(s):
    c = s["case"]
    B, M, L, heads, dim, T = c["B"], c["M"], c["L"], c["heads"], c["dim"], c["block"]
    rows, scales, req = s["rows"], s["scales"], s["req"].long()
    start = s["start"].long()[:, None]
    end = start + s["count"].long()[:, None]
    # The blocks that the new tokens fall into, and the places of each up to the last new token.
    # Windows past the end repeat the last one: they write the same values once more.
    nb = -(-(M + T - 1) // T)
    block = start // T + torch.arange(nb, device="cuda")[None]
    block = torch.minimum(block, (end - 1) // T)  # [B, nb]
    pos = block[:, :, None] * T + torch.arange(T, device="cuda")
    pos = torch.minimum(pos.view(B, nb * T), end - 1)
    new = (pos >= start).view(B, nb, T, 1, 1, 1)
    at = (pos - start).clamp(min=0)
    each = torch.arange(B, device="cuda")[:, None]
    fresh = torch.stack((s["k"][each, at], s["v"][each, at]), dim=2).float()
    fresh = fresh.view(B, nb, T, 2, heads, dim)
    size = torch.where(new & torch.isfinite(fresh), fresh.abs(), torch.zeros_like(fresh))
    peak = size.amax(dim=(2, 5))  # [B, nb, 2, heads]
    begun = (block * T < start)[:, :, None, None]
    was = torch.where(begun, scales[req[:, None], block], torch.zeros_like(peak))
    now = torch.maximum(was, _scale_of(peak, c["code"]))
    wide = now[:, :, None, :, :, None]
    held = rows[req[:, None], pos].view(B, nb, T, 2, heads, dim)
    value = held.view(_code_dtype(c["code"])).float() * was[:, :, None, :, :, None]
    grown = (now > was)[:, :, None, :, :, None]
    again = torch.where(grown, _encode(value, wide, c["code"]), held)
    coded = torch.where(new, _encode(fresh, wide, c["code"]), again)
    rows[req[:, None], pos] = coded.view(B, nb * T, 2 * heads * dim)
    scales[req[:, None], block] = now
    return {"codes": rows.view(_code_dtype(c["code"])), "scales": scales}


def _plain_evict(s):
    c = s["case"]
    B, L, T, heads, dim = c["B"], c["L"], c["block"], c["heads"], c["dim"]
    budget, recent = c["budget"], c["recent"]
    req = s["req"].long()
    n = s["seq_lens"].long().clamp(max=L)[:, None]
    acc = s["acc"][req]
    pos = torch.arange(L, device="cuda")[None]
    # the newest tokens before all, then by weight; those past the end last
    rank = torch.where(pos < n - recent, acc, torch.full_like(acc, math.inf))
    rank = torch.where(pos < n, rank, torch.full_like(acc, -math.inf))
    order = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :budget]
    kept = n.clamp(max=budget)
    slot = torch.arange(budget, device="cuda")[None]
    order = torch.where(slot < kept, order, torch.full_like(order, L))
    order = torch.sort(order, dim=1).values
    keep = torch.where(slot < kept, order, torch.full_like(order, -1))
    held = keep.clamp(min=0)
    kept_acc = torch.where(slot < kept, acc.gather(1, held), torch.zeros_like(acc[:, :budget]))
    blocks = -(-budget // T)
    short = blocks * T - budget
    codes = s["rows"][req[:, None], held].view(_code_dtype(c["code"]))
    value = codes.float().view(B, budget, 2, heads, dim)
    value = value * s["scales"][req[:, None], held // T][..., None]
    value = torch.where((slot < kept)[:, :, None, None, None], value, torch.zeros_like(value))
    value = torch.nn.functional.pad(value, (0, 0, 0, 0, 0, 0, 0, short))
    value = value.view(B, blocks, T, 2, heads, dim)
    size = torch.where(torch.isfinite(value), value.abs(), torch.zeros_like(value))
    scale = _scale_of(size.amax(dim=(2, 5)), c["code"])
    coded = _encode(value, scale[:, :, None, :, :, None], c["code"])
    coded = coded.view(B, blocks * T, 2 * heads * dim)[:, :budget]
    live = slot < kept
    new_rows, new_scales = s["new_rows"], s["new_scales"]
    new_rows.copy_(torch.where(live[:, :, None], coded, new_rows))
    begun = torch.arange(blocks, device="cuda")[None] * T < kept
    new_scales.copy_(torch.where(begun[:, :, None, None], scale, new_scales))
    return {"keep": keep.to(torch.int32), "kept": kept.view(B).to(torch.int32),
            "kept_acc": kept_acc, "codes": new_rows.view(_code_dtype(c["code"])),
            "scales": new_scales}


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    c = case
    heads, dim = c["heads"], c["dim"]
    width = 2 * heads * dim
    if c["op"] == "attend":
        B, S, K, hq = c["B"], c["S"], c["K"], c["heads"] * c["group"]
        live = 0.55 if c["holes"] else 1.0  # mean share of valid entries
        union = _union(S, K)
        # each distinct row and its scales once; the entries; q, out, log-sum-exp, weights and
        # the accumulated weights of the distinct tokens (read and written)
        b = B * union * live * (width + 8 * heads + 8)
        b += B * S * K * 12 + B * S * hq * (4 * dim + 4)
        return {"bytes": b, "flops": 4 * B * S * K * live * hq * dim}
    if c["op"] == "quantize":
        n = c["B"] * c["M"] * (0.75 if c["ragged"] and c["M"] > 1 else 1.0)
        return {"bytes": n * width * 3 + n * 8 * heads / min(c["block"], c["M"]),
                "flops": 3 * n * width}
    n = c["B"] * c["L"] * (0.83 if c["ragged"] else 1.0)
    kept = c["B"] * c["budget"]
    return {"bytes": 4 * n + kept * (8 + 2 * width + 16 * heads / c["block"]),
            "flops": 3 * kept * width}


# ---- the definition in 64 bits ----------------------------------------------------

def _value_table(code):
    """What each of the 256 codes stands for, in 64 bits."""
    if code == "int8":
        return torch.tensor([b - 256 if b > 127 else b for b in range(256)], dtype=torch.float64,
                            device="cuda")
    table = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        if e == 15 and m == 7:
            x = math.nan
        table.append(-x if b > 127 else x)
    return torch.tensor(table, dtype=torch.float64, device="cuda")


def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "quantize": _exact_quantize,
            "evict": _exact_evict}[case["op"]](case, s)


def _exact_attend(c, s):
    table = _value_table(c["code"])
    heads, group, dim = c["heads"], c["group"], c["dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    weights = torch.zeros(s["weights"].shape, dtype=torch.float64, device="cuda")
    acc = s["acc"].double()
    for b in range(c["B"]):
        r = int(s["req"][b])
        for i in range(c["S"]):
            j = torch.nonzero(s["locs"][b, i] >= 0).flatten()
            if not j.numel():
                continue
            x = table[s["rows"][s["locs"][b, i, j].long()].long()].view(-1, 2, heads, dim)
            t = s["topk"][b, i, j].long()
            x = x * s["scales"][r, t // c["block"]].double()[..., None]
            q = s["q"][b, i].double().view(heads, group, dim)
            z = torch.einsum("hgd,khd->hgk", q, x[:, 0]) / math.sqrt(dim)
            top = torch.logsumexp(z, dim=-1)
            p = torch.exp(z - top[..., None])
            out[b, i] = torch.einsum("hgk,khd->hgd", p, x[:, 1]).reshape(heads * group, dim)
            lse[b, i] = top.reshape(-1)
            weights[b, i, j] = p.sum(dim=(0, 1))
            acc[r, t] += weights[b, i, j]
    return {"out": out, "lse": lse, "weights": weights, "acc": acc}


def _exact_scale(peak, code):
    if peak == 0:
        return 0.0
    peak = max(peak, SCALE_FLOOR)
    if code == "int8":
        return peak / INT8_MAX
    e = math.ceil(math.log2(peak / E4M3_MAX))
    e += (math.ldexp(E4M3_MAX, e) < peak) - (math.ldexp(E4M3_MAX, e - 1) >= peak)
    return math.ldexp(1.0, max(e, -100))


def _exact_scales(peaks, code):
    flat = [_exact_scale(p, code) for p in peaks.flatten().tolist()]
    return torch.tensor(flat, dtype=torch.float64, device="cuda").view(peaks.shape)


def _exact_quantize(c, s):
    """Codes as the real values that they round (the int8 ones have to be equal anyway)."""
    table = _value_table(c["code"])
    T, heads, dim = c["block"], c["heads"], c["dim"]
    codes = table[s["rows"].long()]
    scales = s["scales"].double()
    for b in range(c["B"]):
        r, start, count = int(s["req"][b]), int(s["start"][b]), int(s["count"][b])
        x = torch.stack((s["k"][b], s["v"][b]), dim=1).double()  # [M, 2, heads, dim]
        for u in range(start // T, (start + count - 1) // T + 1) if count else ():
            lo, hi = max(start, u * T), min(start + count, (u + 1) * T)
            part = x[lo - start:hi - start]
            scale = _exact_scales(part.abs().amax(dim=(0, 3)), c["code"])
            if lo > u * T:
                was = scales[r, u].clone()
                scale = torch.maximum(was, scale)
                before = codes[r, u * T:lo].view(-1, 2, heads, dim)
                factor = torch.where(scale > 0, was / scale, torch.zeros_like(was))
                codes[r, u * T:lo] = (before * factor[None, ..., None]).view(lo - u * T, -1)
            inv = torch.where(scale > 0, 1.0 / scale, torch.zeros_like(scale))
            codes[r, lo:hi] = (part * inv[None, ..., None]).view(hi - lo, -1)
            scales[r, u] = scale
    return {"codes": None if c["code"] == "int8" else codes, "scales": scales}


def _exact_evict(c, s):
    table = _value_table(c["code"])
    B, T, heads, dim = c["B"], c["block"], c["heads"], c["dim"]
    codes = s["new_rows"].double()
    scales = s["new_scales"].double()
    kept_acc = s["kept_acc"].double() * 0
    for b in range(B):
        r, n = int(s["req"][b]), min(int(s["seq_lens"][b]), c["L"])
        w = s["acc"][r, :n].double()
        if n <= c["budget"]:
            keep = torch.arange(n, device="cuda")
        else:
            old = n - c["recent"]
            heavy = torch.argsort(w[:old], descending=True, stable=True)
            heavy = heavy[:c["budget"] - c["recent"]]
            keep = torch.cat((heavy, torch.arange(old, n, device="cuda"))).sort().values
        kept_acc[b, :keep.numel()] = w[keep]
        x = table[s["rows"][r, keep].long()].view(-1, 2, heads, dim)
        x = x * s["scales"][r, keep // T].double()[..., None]
        part = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, 0, 0, -x.shape[0] % T))
        part = part.view(-1, T, 2, heads, dim)
        scale = _exact_scales(part.abs().amax(dim=(1, 4)), c["code"])
        scales[b, :scale.shape[0]] = scale
        inv = torch.where(scale > 0, 1.0 / scale, torch.zeros_like(scale))
        part = (part * inv[:, None, ..., None]).reshape(-1, 2 * heads * dim)
        codes[b, :keep.numel()] = part[:keep.numel()]
    return {"keep": None, "kept": None, "kept_acc": kept_acc,
            "codes": None if c["code"] == "int8" else codes, "scales": scales}
