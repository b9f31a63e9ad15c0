"""Plain implementation of the 8-bit key/value row calls: attention, weights
and eviction in 64 bits; codes and scales in the 32-bit operations that the
header defines, so that they can be compared bit for bit."""
import math

import numpy as np
import torch


def decode_table(code: str) -> np.ndarray:
    """What each of the 256 codes stands for."""
    if code == "int8":
        return np.arange(256, dtype=np.uint8).view(np.int8).astype(np.float64)
    out = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[b] = math.nan if (e, m) == (15, 7) else x
        if b >= 128:
            out[b] = -out[b]
    return out


def unpack(rows: np.ndarray, heads: int, dim: int, code: str) -> np.ndarray:
    """[..., W] bytes -> [..., 2, heads, dim] values without their scales."""
    x = decode_table(code)[rows[..., :2 * heads * dim]]
    return x.reshape(rows.shape[:-1] + (2, heads, dim))


def attend(q, rows, locs, topk, req, scales, T, L, heads, code, sm_scale):
    """Outputs in 64 bits, and the sums that error bounds are made of."""
    B, S, Hq, D = q.shape
    K = locs.shape[2]
    G = Hq // heads
    out = np.zeros((B, S, Hq, D))
    spread = np.zeros((B, S, Hq, D))      # sum of p |v|
    lse = np.full((B, S, Hq), -np.inf)
    logit = np.zeros((B, S, Hq))          # largest sum of |q k| over the entries
    biggest = np.zeros((B, S, Hq, D))     # largest |v|
    weights = np.zeros((B, S, K))
    for b in range(B):
        if not 0 <= req[b] < scales.shape[0]:
            continue
        for s in range(S):
            ok = ((locs[b, s] >= 0) & (locs[b, s] < rows.shape[0]) & (topk[b, s] >= 0)
                  & (topk[b, s] < L))
            j = np.nonzero(ok)[0]
            if j.size == 0:
                continue
            x = unpack(rows[locs[b, s, j]], heads, D, code)
            x = x * scales[req[b], topk[b, s, j] // T].astype(np.float64)[..., None]
            for i in range(Hq):
                k, v = x[:, 0, i // G], x[:, 1, i // G]
                z = (k @ q[b, s, i]) * sm_scale
                logit[b, s, i] = (np.abs(k) @ np.abs(q[b, s, i])).max() * abs(sm_scale)
                lse[b, s, i] = z.max() + np.log(np.exp(z - z.max()).sum())
                p = np.exp(z - lse[b, s, i])
                out[b, s, i] = p @ v
                spread[b, s, i] = p @ np.abs(v)
                biggest[b, s, i] = np.abs(v).max(axis=0)
                weights[b, s, j] += p
    return {"out": out, "spread": spread, "lse": lse, "logit": logit, "weights": weights,
            "biggest": biggest}


def scale_of(peak: torch.Tensor, code: str) -> torch.Tensor:
    big = peak.clamp(min=2.0 ** -100)
    if code == "e4m3":
        frac, e = torch.frexp(big)  # frac in [0.5, 1); 448 = 0.875 * 2^9
        e = torch.where(frac <= 0.875, e - 9, e - 8).clamp(min=-100)
        s = torch.ldexp(torch.ones_like(big), e)
    else:
        s = big / torch.full_like(big, 127.0)
    return torch.where(peak > 0, s, torch.zeros_like(s))


def encode(x: torch.Tensor, scale: torch.Tensor, code: str) -> torch.Tensor:
    r = torch.where(scale > 0, torch.reciprocal(scale), torch.zeros_like(scale))
    y = x * r
    if code == "e4m3":
        return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    y = torch.where(torch.isnan(y), torch.zeros_like(y), y)
    return torch.round(y).clamp(-127, 127).to(torch.int8).view(torch.uint8)


def peak_of(x: torch.Tensor, dims) -> torch.Tensor:
    return torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(dim=dims)


def quantize(k, v, req, start, count, rows, scales, T, code):
    """In place on rows uint8 [R, L, W] and scales fp32 [R, NB, 2, heads] (CPU tensors)."""
    B, M, heads, D = k.shape
    R, L, _ = rows.shape
    kind = torch.float8_e4m3fn if code == "e4m3" else torch.int8
    for b in range(B):
        q, p, n = int(req[b]), int(start[b]), int(count[b])
        if not 0 <= q < R or p < 0 or n < 0 or n > M or p + n > L or n == 0:
            continue
        x = torch.stack((k[b, :n], v[b, :n]), dim=1).float()  # [n, 2, heads, D]
        for u in range(p // T, (p + n - 1) // T + 1):
            lo, hi = max(p, u * T), min(p + n, (u + 1) * T)
            part = x[lo - p:hi - p]
            now = scale_of(peak_of(part, (0, 3)), code)
            if lo > u * T:
                was = scales[q, u].clone()
                now = torch.maximum(was, now)
                held = rows[q, u * T:lo, :2 * heads * D]
                old = held.view(kind).float().view(-1, 2, heads, D) * was[None, ..., None]
                again = encode(old, now[None, ..., None].expand_as(old), code)
                grown = (now > was)[None, ..., None]
                again = torch.where(grown, again, held.reshape(again.shape))
                rows[q, u * T:lo, :2 * heads * D] = again.reshape(lo - u * T, -1)
            coded = encode(part, now[None, ..., None].expand_as(part), code)
            rows[q, lo:hi, :2 * heads * D] = coded.reshape(hi - lo, -1)
            scales[q, u] = now


def evict(acc, req, seq_lens, recent, budget):
    """keep [B, budget], kept [B], kept_acc [B, budget] as numpy arrays."""
    R, L = acc.shape
    B = len(req)
    keep = np.full((B, budget), -1, np.int32)
    kept = np.zeros(B, np.int32)
    kept_acc = np.zeros((B, budget), np.float32)
    for b in range(B):
        n = min(int(seq_lens[b]), L)
        if not 0 <= req[b] < R or n <= 0:
            continue
        w = acc[req[b], :n]
        if n <= budget:
            pos = np.arange(n)
        else:
            m = n - recent
            key = np.where(np.isnan(w[:m]), -np.inf, w[:m]).astype(np.float64)
            nan_last = np.isnan(w[:m])
            order = np.lexsort((np.arange(m), nan_last, -key))
            pos = np.sort(np.concatenate((order[:budget - recent], np.arange(m, n))))
        kept[b] = pos.size
        keep[b, :pos.size] = pos
        kept_acc[b, :pos.size] = w[pos]
    return keep, kept, kept_acc


def compact(src, src_scales, src_req, keep, kept, dst, dst_scales, dst_req, T, heads, D, code):
    """In place on dst and dst_scales (CPU tensors)."""
    kind = torch.float8_e4m3fn if code == "e4m3" else torch.int8
    width = 2 * heads * D
    for b in range(len(src_req)):
        q, r = int(src_req[b]), int(dst_req[b])
        n = min(int(kept[b]), keep.shape[1], dst.shape[1])
        if not 0 <= q < src.shape[0] or not 0 <= r < dst.shape[0] or n <= 0:
            continue
        pos = keep[b, :n].long()
        ok = (pos >= 0) & (pos < src.shape[1])
        at = pos.clamp(0, src.shape[1] - 1)
        x = src[q, at, :width].view(kind).float().view(n, 2, heads, D)
        x = x * src_scales[q, at // T][..., None]
        x = torch.where(ok[:, None, None, None], x, torch.zeros_like(x))
        for u in range((n + T - 1) // T):
            part = x[u * T:(u + 1) * T]
            now = scale_of(peak_of(part, (0, 3)), code)
            coded = encode(part, now[None, ..., None].expand_as(part), code)
            dst[r, u * T:u * T + part.shape[0], :width] = coded.reshape(part.shape[0], -1)
            dst_scales[r, u] = now
