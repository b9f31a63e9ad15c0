"""Cases of the operators around a swap-in: per-head norms and position rotation of
new queries and keys, block selection by bounds on the keys (with the upkeep
of the bounds), and attention over a prefix that requests of a batch share.

``own`` selects the framework's calls; otherwise the same results come from
elementary torch operations in 32 bits (angles, and scores that decide a
selection, in 64).
"""
import functools
import math

import torch

own = False


# ---- the cases ----------------------------------------------------------------

def _rotate(name, B, M, heads, group, dim, rot, axes, adjacent, norm, dtype, far):
    return dict(name=name, op="rotate", B=B, M=M, heads=heads, group=group, dim=dim, rot=rot,
                axes=axes, adjacent=adjacent, norm=norm, dtype=dtype, far=far)


def _bound(name, B, M, L, heads, dim, block, dtype, ragged):
    return dict(name=name, op="bound", B=B, M=M, L=L, heads=heads, dim=dim, block=block,
                dtype=dtype, ragged=ragged)


def _select(name, B, S, L, heads, group, dim, block, blocks, first, last, dtype, ragged):
    return dict(name=name, op="select", B=B, S=S, L=L, heads=heads, group=group, dim=dim,
                block=block, blocks=blocks, first=first, last=last, dtype=dtype, ragged=ragged)


def _prefix(name, B, S, groups, L, heads, group, dim, block, dtype, code, ragged, join):
    return dict(name=name, op="prefix", B=B, S=S, groups=groups, L=L, heads=heads, group=group,
                dim=dim, block=block, dtype=dtype, code=code, ragged=ragged, join=join)


def listed():
    return [
        # One decoded token for each of 64 requests: latency counts.
        _rotate("rotate_token", 64, 1, 8, 8, 128, 128, 1, False, True, "bf16", 32768),
        # Prompts of 8192 tokens: bandwidth counts.
        _rotate("rotate_prompt", 4, 8192, 8, 4, 128, 128, 1, False, True, "bf16", 8192),
        # Chunks of image and text tokens: positions in time, height and width, half of each
        # head rotated in adjacent pairs; odd sizes.
        _rotate("rotate_three_axes", 6, 777, 5, 3, 96, 48, 3, True, True, "fp16", 131072),
        # One decoded token for each of 64 requests, into blocks that are still filling.
        _bound("bound_token", 64, 1, 32768, 8, 128, 64, "bf16", True),
        # Prompts of 8192 tokens: whole blocks.
        _bound("bound_prompt", 4, 8192, 8192, 8, 128, 64, "bf16", False),
        # One request over a 4096-token sequence: 32 of 256 blocks.
        _select("select_one_request", 1, 1, 4096, 2, 4, 128, 16, 32, 1, 2, "bf16", False),
        # A full decode batch: 2048 tokens of 32768, in blocks of 64.
        _select("select_decode_batch", 64, 1, 32768, 8, 8, 128, 64, 32, 1, 2, "bf16", False),
        # Four steps of multi-token prediction over long contexts of different lengths.
        _select("select_long_four_steps", 12, 4, 131072, 4, 6, 96, 32, 64, 1, 4, "fp16", True),
        # A few requests behind a short common prompt: the smallest call.
        _prefix("prefix_few_requests", 4, 1, 1, 512, 2, 4, 128, 64, "bf16", "e4m3", False, True),
        # A decode batch behind one common prompt of 32768 tokens: the products count.
        _prefix("prefix_decode_batch", 64, 1, 1, 32768, 8, 8, 128, 64, "bf16", "e4m3", False,
                True),
        # Two requests over a very long document: bandwidth counts.
        _prefix("prefix_long_document", 2, 1, 1, 131072, 8, 4, 128, 64, "bf16", "e4m3", False,
                False),
        # Three prompts of different lengths in one batch, 3 steps, int8 codes, odd sizes.
        _prefix("prefix_three_prompts_int8", 21, 3, 3, 9973, 5, 3, 96, 48, "fp16", "int8", True,
                True),
    ]


def _spread(rng, low, high):
    """A whole number from low to high, spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["rotate", "bound", "select", "select", "prefix", "prefix"])
    dim = rng.choice([64, 96, 128, 128, 192, 256])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    heads = rng.choice([1, 2, 3, 4, 5, 8, 8, 12])
    while heads * dim > 1024:
        heads = rng.choice([1, 2, 3, 4, 5, 8])
    group = rng.choice([1, 2, 3, 4, 6, 8, 8, 12, 16])
    while heads * group > 64:
        group = rng.choice([1, 2, 3, 4, 6, 8])
    width = heads * dim
    if op == "rotate":
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        M = _spread(rng, 1, 8192)
        most = 4 * 8192 * 5120 // (M * width * (group + 1) * (2 if dtype == "fp32" else 1))
        B = _spread(rng, 1, max(1, min(64, most)))
        axes = rng.choice([1, 1, 2, 3])
        rot = dim if rng.random() < 0.6 else max(16, dim // 32 * 16)
        c = _rotate("", B, M, heads, group, dim, rot, axes, rng.random() < 0.4, rng.random() < 0.8,
                    dtype, _spread(rng, 64, 1 << 20))
    elif op == "bound":
        M = _spread(rng, 1, 8192)
        B = _spread(rng, 1, max(1, min(64, 4 * 8192 * 1024 // (M * width))))
        c = _bound("", B, M, M + rng.randrange(1, 512), heads, dim,
                   rng.choice([8, 16, 32, 48, 64, 128]), dtype, rng.random() < 0.6)
    elif op == "select":
        block = rng.choice([16, 32, 48, 64, 128])
        S = rng.choice([1, 1, 2, 3, 4])
        L = _spread(rng, 64, 131072)
        blocks = _spread(rng, 1, max(1, min(8192 // (S * block), -(-L // block))))
        B = _spread(rng, 1, max(1, min(64, 64 * 512 * 1024 * block // (L * width))))
        first = min(blocks, rng.choice([0, 1, 1, 2]))
        last = min(blocks - first, rng.choice([0, 1, 2, 4]))
        c = _select("", B, S, L, heads, group, dim, block, blocks, first, last, dtype,
                    rng.random() < 0.5)
    else:
        S = rng.choice([1, 1, 2, 3, 4])
        L = _spread(rng, 64, 131072)
        most = max(1, min(64, 64 * 64 * 32768 * 128 // (S * heads * group * dim * L)))
        B = _spread(rng, 1, most)
        groups = min(B, rng.choice([1, 1, 2, 3, 5]), max(1, 131072 * 1024 // (L * width)))
        c = _prefix("", B, S, groups, L, heads, group, dim, rng.choice([16, 32, 48, 64, 128, 256]),
                    dtype, rng.choice(["e4m3", "e4m3", "int8"]), rng.random() < 0.6,
                    rng.random() < 0.7)
    del c["name"]
    return c


# ---- inputs ---------------------------------------------------------------------

def _torch_dtype(name):
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    return {"rotate": _prepare_rotate, "bound": _prepare_bound, "select": _prepare_select,
            "prefix": _prepare_prefix}[case["op"]](case, gen, s)


def _channels(heads, dim, gen):
    """Channels differ in size, as those of keys do."""
    return torch.exp(0.5 * torch.randn((heads, dim), device="cuda", generator=gen))


def _frequencies(c):
    """Angle per position and pair (64 bits), and the axis that turns a pair."""
    pairs = c["rot"] // 2
    freq = [10000.0 ** (-j / pairs) for j in range(pairs)]
    axis = [j * c["axes"] // pairs for j in range(pairs)]
    return freq, axis


def _prepare_rotate(c, gen, s):
    B, M, heads, dim, t = c["B"], c["M"], c["heads"], c["dim"], _torch_dtype(c["dtype"])
    # the new queries, keys and values of a token lie side by side, as one projection writes them
    hq = heads * c["group"]
    x = torch.empty((B, M, hq + 2 * heads, dim), dtype=t, device="cuda")
    size = _channels(hq + 2 * heads, dim, gen)
    for b in range(B):
        x[b] = (torch.randn(x.shape[1:], device="cuda", generator=gen) * size).to(t)
    s["q"], s["k"] = x[:, :, :hq], x[:, :, hq:hq + heads]
    s["q_out"] = torch.empty((B, M, hq, dim), dtype=t, device="cuda")
    s["k_out"] = torch.empty((B, M, heads, dim), dtype=t, device="cuda")
    s["q_weight"] = s["k_weight"] = None
    if c["norm"]:
        s["q_weight"] = 1.0 + 0.2 * torch.randn(dim, device="cuda", generator=gen)
        s["k_weight"] = 1.0 + 0.2 * torch.randn(dim, device="cuda", generator=gen)
    start = torch.rand((c["axes"], B, 1), device="cuda", generator=gen, dtype=torch.float64)
    start = (start * max(1, c["far"] - M)).long()
    if c["axes"] == 1:
        s["pos"] = (start + torch.arange(M, device="cuda")).to(torch.int32)
    else:  # patches of images: rows and columns start anew in every image
        at = torch.arange(M, device="cuda")
        side = max(1, int(math.sqrt(M)))
        step = [at // (side * side), at // side % side, at % side][3 - c["axes"]:]
        s["pos"] = (start + torch.stack(step)[:, None]).to(torch.int32)
    if own:
        import sparse_attention_kv_swap_gb300 as hs
        freq, axis = _frequencies(c)
        s["rope"] = hs.make_rope(freq, axis, adjacent=c["adjacent"])
    return s


def _prepare_bound(c, gen, s):
    B, M, L, heads, dim, T = c["B"], c["M"], c["L"], c["heads"], c["dim"], c["block"]
    t = _torch_dtype(c["dtype"])
    size = _channels(heads, dim, gen)
    s["k"] = (torch.randn((B, M, heads, dim), device="cuda", generator=gen) * size).to(t)
    s["bounds"] = _bounds(B, -(-L // T), heads, dim, t, gen)
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


def _bounds(R, NB, heads, dim, dtype, gen):
    """Bounds as blocks of keys have them: a common centre, the block's own shift, and its
    spread."""
    size = _channels(heads, dim, gen)
    centre = torch.randn((heads, dim), device="cuda", generator=gen) * size
    out = torch.empty((R, NB, heads, 2, dim), dtype=dtype, device="cuda")
    for r in range(R):
        mid = centre + 0.5 * size * torch.randn((NB, heads, dim), device="cuda", generator=gen)
        wide = size * (1.0 + torch.rand((NB, heads, dim), device="cuda", generator=gen))
        out[r, :, :, 0] = (mid - wide).to(dtype)
        out[r, :, :, 1] = (mid + wide).to(dtype)
    return out


def _prepare_select(c, gen, s):
    B, S, L, heads, dim, T = c["B"], c["S"], c["L"], c["heads"], c["dim"], c["block"]
    t = _torch_dtype(c["dtype"])
    s["q"] = torch.randn((B, S, heads * c["group"], dim), device="cuda", generator=gen).to(t)
    s["bounds"] = _bounds(B, -(-L // T), heads, dim, t, gen)
    s["req"] = torch.randperm(B, device="cuda", generator=gen).to(torch.int32)
    n = torch.full((B,), float(L), device="cuda")
    if c["ragged"]:
        n = L - (torch.rand(B, device="cuda", generator=gen) * (L // 2)).floor()
    s["seq_lens"] = n.to(torch.int32)
    s["topk"] = torch.empty((B, S, c["blocks"] * T), dtype=torch.int32, device="cuda")
    s["blocks"] = torch.empty((B, S, c["blocks"]), dtype=torch.int32, device="cuda")
    s["scores"] = torch.empty((B, S, -(-L // T)), device="cuda")
    if own:
        import sparse_attention_kv_swap_gb300 as hs
        s["workspace"] = torch.empty(hs.hs_select_workspace_bytes(B, S, L, T), dtype=torch.uint8,
                                     device="cuda")
    return s


def _prepare_prefix(c, gen, s):
    B, S, G, L, heads, dim, T = (c[x] for x in ("B", "S", "groups", "L", "heads", "dim", "block"))
    hq, t = heads * c["group"], _torch_dtype(c["dtype"])
    s["q"] = torch.randn((B, S, hq, dim), device="cuda", generator=gen).to(t)
    s["rows"] = torch.empty((G, L, 2 * heads * dim), dtype=torch.uint8, device="cuda")
    for g in range(G):
        x = torch.randn((L, 2 * heads * dim), device="cuda", dtype=torch.float16, generator=gen)
        if c["code"] == "e4m3":
            x = x.mul_(90.0).clamp_(-440.0, 440.0).to(torch.float8_e4m3fn)
        else:
            x = x.mul_(32.0).round_().clamp_(-127.0, 127.0).to(torch.int8)
        s["rows"][g] = x.view(torch.uint8)
    shape = (G, -(-L // T), 2, heads)
    if c["code"] == "e4m3":
        e = torch.randint(-8, -5, shape, device="cuda", generator=gen)
        s["scales"] = torch.ldexp(torch.ones(shape, device="cuda"), e)
    else:
        s["scales"] = torch.rand(shape, device="cuda", generator=gen) * 0.06 + 0.015
    s["prefix"] = torch.randperm(G, device="cuda", generator=gen).to(torch.int32)
    n = torch.full((G,), float(L), device="cuda")
    starts = torch.arange(G + 1, device="cuda") * B // G
    if c["ragged"]:
        n = L - (torch.rand(G, device="cuda", generator=gen) * (0.7 * L)).floor()
        cuts = (torch.rand(G - 1, device="cuda", generator=gen) * (B + 1)).floor().long()
        starts[1:G] = cuts.sort().values
    s["lens"], s["starts"] = n.to(torch.int32), starts.to(torch.int32)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((B, S, hq), device="cuda")
    s["join_out"] = s["join_lse"] = None
    if c["join"]:  # the attention over the requests' own tokens, some without any
        s["join_out"] = (0.1 * torch.randn((B, S, hq, dim), device="cuda", generator=gen)).to(t)
        lse = math.log(L) + torch.randn((B, S, hq), device="cuda", generator=gen)
        none = torch.rand((B, S, 1), device="cuda", generator=gen) < 0.05
        s["join_lse"] = lse.masked_fill(none, -math.inf)
        s["join_out"] = s["join_out"].masked_fill(none[..., None], 0.0)
    if own:
        import sparse_attention_kv_swap_gb300 as hs
        fmt = _format(heads, dim, T, c["code"])
        need = hs.hs_prefix_workspace_bytes(fmt, B, S, hq, G)
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
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
        return {"rotate": _own_rotate, "bound": _own_bound, "select": _own_select,
                "prefix": _own_prefix}[op](s)
    return {"rotate": _plain_rotate, "bound": _plain_bound, "select": _plain_select,
            "prefix": _plain_prefix}[op](s)


def _own_rotate(s):
    import sparse_attention_kv_swap_gb300 as hs
    hs.hs_norm_rope(s["q"], s["k"], s["pos"], s["rope"], s["q_out"], s["k_out"],
                    q_weight=s["q_weight"], k_weight=s["k_weight"])
    return {"q": s["q_out"], "k": s["k_out"]}


def _own_bound(s):
    import sparse_attention_kv_swap_gb300 as hs
    c = s["case"]
    hs.hs_bound_keys(s["k"], s["req"], s["start"], s["count"], c["block"], c["L"], s["bounds"])
    return {"bounds": s["bounds"]}


def _own_select(s):
    import sparse_attention_kv_swap_gb300 as hs
    c = s["case"]
    hs.hs_select_blocks(s["q"], s["bounds"], s["req"], s["seq_lens"], c["block"], c["L"],
                        c["first"], c["last"], s["blocks"], s["topk"], s["scores"],
                        workspace=s["workspace"])
    return {"blocks": s["blocks"], "topk": s["topk"], "scores": s["scores"]}


def _own_prefix(s):
    import sparse_attention_kv_swap_gb300 as hs
    c = s["case"]
    fmt = _format(c["heads"], c["dim"], c["block"], c["code"])
    hs.hs_attend_prefix(fmt, s["q"], s["rows"], s["scales"], s["prefix"], s["lens"], s["starts"],
                        s["out"], lse=s["lse"], join_out=s["join_out"], join_lse=s["join_lse"],
                        workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def _plain_rotate(s):
    c = s["case"]
    freq, axis = _frequencies(c)
    freq = torch.tensor(freq, dtype=torch.float64, device="cuda")
    axis = torch.tensor(axis, device="cuda")
    angle = s["pos"][axis].permute(1, 2, 0).double() * freq  # [B, M, rot / 2]
    cos, sin = torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]
    rot, half = c["rot"], c["rot"] // 2

    def turned(x, weight, out):
        y = x.float()
        if weight is not None:
            y = y * torch.rsqrt((y * y).mean(dim=-1, keepdim=True) + 1e-6) * weight
        if c["adjacent"]:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            z = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
        else:
            a, b = y[..., :half], y[..., half:rot]
            z = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
        out[..., :rot] = z.to(out.dtype)
        out[..., rot:] = y[..., rot:].to(out.dtype)
        return out

    return {"q": turned(s["q"], s["q_weight"], s["q_out"]),
            "k": turned(s["k"], s["k_weight"], s["k_out"])}


def _plain_bound(s):
    c = s["case"]
    B, M, heads, dim, T = c["B"], c["M"], c["heads"], c["dim"], c["block"]
    bounds, req = s["bounds"], s["req"].long()
    start = s["start"].long()[:, None]
    end = start + s["count"].long()[:, None]
    # The blocks that the new tokens fall into, and the places of each up to the last new token.
    # Windows past the end repeat the last one: they write the same values once more.
    nb = -(-(M + T - 1) // T)
    block = torch.minimum(start // T + torch.arange(nb, device="cuda")[None], (end - 1) // T)
    pos = block[:, :, None] * T + torch.arange(T, device="cuda")
    pos = torch.minimum(pos.view(B, nb * T), end - 1)
    new = (pos >= start).view(B, nb, T, 1, 1)
    each = torch.arange(B, device="cuda")[:, None]
    x = s["k"][each, (pos - start).clamp(min=0)].float().view(B, nb, T, heads, dim)
    low = torch.where(new, x, torch.full_like(x, math.inf)).amin(dim=2)
    high = torch.where(new, x, torch.full_like(x, -math.inf)).amax(dim=2)
    begun = (block * T < start)[:, :, None, None]
    was = bounds[req[:, None], block].float()
    low = torch.where(begun, torch.minimum(low, was[:, :, :, 0]), low)
    high = torch.where(begun, torch.maximum(high, was[:, :, :, 1]), high)
    bounds[req[:, None], block] = torch.stack((low, high), dim=3).to(bounds.dtype)
    return {"bounds": bounds}


def _plain_select(s):
    c = s["case"]
    B, S, heads, group, dim, T = (c[x] for x in ("B", "S", "heads", "group", "dim", "block"))
    q = s["q"].double().view(B, S, heads, group, dim)
    up, down = q.clamp(min=0).sum(dim=3), q.clamp(max=0).sum(dim=3)
    x = s["bounds"][s["req"].long()].double()  # [B, NB, heads, 2, dim]
    score = torch.einsum("bshd,bnhd->bsn", up, x[:, :, :, 1])
    score += torch.einsum("bshd,bnhd->bsn", down, x[:, :, :, 0])
    n = s["seq_lens"].long().clamp(max=c["L"])[:, None, None]
    nb = (n + T - 1) // T
    at = torch.arange(score.shape[2], device="cuda")
    s["scores"].copy_(torch.where(at < nb, score, -math.inf))
    rank = torch.where((at < c["first"]) | (at >= nb - c["last"]), math.inf, score)
    rank = torch.where(at < nb, rank, -math.inf)
    order = torch.sort(rank, dim=2, descending=True, stable=True).indices[..., :c["blocks"]]
    slot = torch.arange(c["blocks"], device="cuda")
    order = torch.where(slot < nb, order, at.numel()).sort(dim=2).values
    blocks = torch.where(slot < nb, order, -1)
    token = blocks[..., None] * T + torch.arange(T, device="cuda")
    token = torch.where((blocks[..., None] >= 0) & (token < n[..., None]), token, -1)
    s["blocks"].copy_(blocks)
    s["topk"].copy_(token.view(B, S, -1))
    return {"blocks": s["blocks"], "topk": s["topk"], "scores": s["scores"]}


def _plain_prefix(s):
    c = s["case"]
    B, S, heads, group, dim, T = (c[x] for x in ("B", "S", "heads", "group", "dim", "block"))
    kind = torch.float8_e4m3fn if c["code"] == "e4m3" else torch.int8
    q = s["q"].float().view(B, S, heads, group, dim)
    out = torch.zeros((B, S, heads, group, dim), device="cuda")
    lse = torch.full((B, S, heads, group), -math.inf, device="cuda")
    starts, lens = s["starts"].tolist(), s["lens"].tolist()
    for g, r in enumerate(s["prefix"].tolist()):
        lo, hi, n = starts[g], starts[g + 1], lens[g]
        block = torch.arange(n, device="cuda") // T
        for h in range(heads if hi > lo and n > 0 else 0):
            k, v = (s["rows"][r, :n, at:at + dim].view(kind).float()
                    for at in (h * dim, (heads + h) * dim))
            k = k * s["scales"][r, block, 0, h, None]
            v = v * s["scales"][r, block, 1, h, None]
            z = torch.matmul(q[lo:hi, :, h].reshape(-1, dim) * dim ** -0.5, k.t())
            top = z.amax(dim=1, keepdim=True)
            z = z.sub_(top).exp_()
            total = z.sum(dim=1, keepdim=True)
            out[lo:hi, :, h] = (torch.matmul(z, v) / total).view(hi - lo, S, group, dim)
            lse[lo:hi, :, h] = (top + torch.log(total)).view(hi - lo, S, group)
    out, lse = out.view(B, S, -1, dim), lse.view(B, S, -1)
    if c["join"]:
        both = torch.logaddexp(lse, s["join_lse"])
        safe = torch.where(both == -math.inf, torch.zeros_like(both), both)
        out = (out * torch.exp(lse - safe)[..., None]
               + s["join_out"].float() * torch.exp(s["join_lse"] - safe)[..., None])
        lse = both
    return {"out": out.to(s["q"].dtype), "lse": lse}


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    c = case
    heads, dim = c["heads"], c["dim"]
    size = 4 if c["dtype"] == "fp32" else 2
    if c["op"] == "rotate":
        n = c["B"] * c["M"]
        each = heads * (c["group"] + 1) * dim
        return {"bytes": n * (2 * size * each + 4 * c["axes"]),
                "flops": n * each * (4 * c["norm"] + 3 * c["rot"] / dim)}
    if c["op"] == "bound":
        part = 0.75 if c["ragged"] and c["M"] > 1 else 1.0
        n = c["B"] * c["M"] * part
        touched = c["B"] * (c["M"] * part / c["block"] if c["M"] > c["block"] else 1)
        return {"bytes": size * heads * dim * (n + 2 * touched), "flops": 2 * n * heads * dim}
    if c["op"] == "select":
        B, S, hq = c["B"], c["S"], heads * c["group"]
        blocks = B * c["L"] / c["block"] * (0.75 if c["ragged"] else 1.0)
        b = blocks * heads * 2 * dim * size + B * S * (hq * dim * size)
        b += B * S * 4 * c["L"] / c["block"]
        return {"bytes": b + B * S * c["blocks"] * 4 * (c["block"] + 1),
                "flops": 4 * S * blocks * heads * dim + 2 * B * S * hq * dim}
    B, S, hq = c["B"], c["S"], heads * c["group"]
    n = c["L"] * (0.65 if c["ragged"] else 1.0)
    b = c["groups"] * n * (2 * heads * dim + 8 * heads / c["block"])
    b += B * S * hq * (dim * size + 4) * (2 if c["join"] else 1) + B * S * hq * dim * size
    return {"bytes": b, "flops": 4 * B * S * hq * n * dim}


# ---- the definition in 64 bits ----------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"rotate": _exact_rotate, "bound": _exact_bound, "select": _exact_select,
            "prefix": _exact_prefix}[case["op"]](case, s)


def _exact_rotate(c, s):
    freq, axis = _frequencies(c)
    got = {}
    for name in ("q", "k"):
        x = s[name].double()
        if c["norm"]:
            x = x / torch.sqrt((x ** 2).sum(dim=-1, keepdim=True) / c["dim"] + 1e-6)
            x = x * s[name + "_weight"].double()
        y = x.clone()
        for j, f in enumerate(freq):
            i0, i1 = (2 * j, 2 * j + 1) if c["adjacent"] else (j, j + c["rot"] // 2)
            # one complex number per pair, turned by e^(i angle)
            turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                               s["pos"][axis[j]].double() * f)[..., None]
            z = torch.complex(x[..., i0], x[..., i1]) * turn
            y[..., i0], y[..., i1] = z.real, z.imag
        got[name] = y
    return got


def _exact_bound(c, s):
    T = c["block"]
    bounds = s["bounds"].double()
    for b in range(c["B"]):
        r, start, count = int(s["req"][b]), int(s["start"][b]), int(s["count"][b])
        for u in range(start // T, (start + count - 1) // T + 1) if count else ():
            lo, hi = max(start, u * T), min(start + count, (u + 1) * T)
            part = s["k"][b, lo - start:hi - start].double()
            if lo > u * T:
                part = torch.cat((part, bounds[r, u].transpose(0, 1)))
            bounds[r, u, :, 0], bounds[r, u, :, 1] = part.amin(dim=0), part.amax(dim=0)
    return {"bounds": bounds}


def _exact_select(c, s):
    """A block's score is the sum over query heads and channels of the larger of the products of
    a query element with the two bounds."""
    scores = torch.full(s["scores"].shape, -math.inf, dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        nb = -(-min(int(s["seq_lens"][b]), c["L"]) // c["block"])
        x = s["bounds"][int(s["req"][b]), :nb].double()
        for i in range(c["heads"] * c["group"]):
            low, high = x[:, i // c["group"], 0], x[:, i // c["group"], 1]
            for j in range(c["S"]):
                q = s["q"][b, j, i].double()
                part = torch.maximum(low * q, high * q).sum(dim=1)
                scores[b, j, :nb] = part if i == 0 else scores[b, j, :nb] + part
    return {"blocks": None, "topk": None, "scores": scores}


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


def _exact_prefix(c, s):
    if work(c)["flops"] > 1.2e10:
        return None  # minutes in 64 bits
    B, S, heads, group, dim, T = (c[x] for x in ("B", "S", "heads", "group", "dim", "block"))
    table = _value_table(c["code"])
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    for g in range(c["groups"]):
        r, n = int(s["prefix"][g]), int(s["lens"][g])
        lo, hi = int(s["starts"][g]), int(s["starts"][g + 1])
        scale = s["scales"][r].double().repeat_interleave(T, dim=0)[:n]  # [n, 2, heads]
        for i in range(heads * group if hi > lo and n > 0 else 0):
            h = i // group
            code = s["rows"][r, :n].long()
            k = table[code[:, h * dim:(h + 1) * dim]] * scale[:, 0, h, None]
            v = table[code[:, (heads + h) * dim:(heads + h + 1) * dim]] * scale[:, 1, h, None]
            z = torch.einsum("bsd,kd->bsk", s["q"][lo:hi, :, i].double(), k) / math.sqrt(dim)
            lse[lo:hi, :, i] = torch.logsumexp(z, dim=-1)
            out[lo:hi, :, i] = torch.einsum("bsk,kd->bsd", torch.softmax(z, dim=-1), v)
    if c["join"]:
        other = s["join_lse"].double()
        top = torch.maximum(lse, other)
        top = torch.where(top == -math.inf, torch.zeros_like(top), top)
        a, b = torch.exp(lse - top)[..., None], torch.exp(other - top)[..., None]
        both = a + b
        out = torch.where(both > 0, (a * out + b * s["join_out"].double()) / both,
                          torch.zeros_like(out))
        lse = top + torch.log(both[..., 0])
    return {"out": out, "lse": lse}
