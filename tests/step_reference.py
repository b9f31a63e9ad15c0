"""Plain implementation, in 64 bits, of the calls around a decode step: norms and
rotation, bounds and selection of key blocks, attention over shared prefixes."""
import numpy as np

import kv_reference as ref


def norm_rope(x, weight, eps, pos, freq, axis, adjacent):
    """x [B, M, H, D]; pos [axes, B, M]; freq and axis [rot / 2].  Returns the outputs and the
    length of each element's pair (its own magnitude where it does not turn)."""
    x = x.astype(np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps) * weight.astype(np.float64)
    y, size = x.copy(), np.abs(x)
    for j, f in enumerate(freq):
        i0, i1 = (2 * j, 2 * j + 1) if adjacent else (j, j + len(freq))
        angle = pos[axis[j]].astype(np.float64) * f
        c, s = np.cos(angle)[..., None], np.sin(angle)[..., None]
        y[..., i0] = x[..., i0] * c - x[..., i1] * s
        y[..., i1] = x[..., i0] * s + x[..., i1] * c
        size[..., i0] = size[..., i1] = np.hypot(x[..., i0], x[..., i1])
    return y, size


def bound(k, req, start, count, T, L, bounds):
    """In place on bounds [R, NB, H, 2, D] (float64 values of the keys' type)."""
    M = k.shape[1]
    for b in range(len(req)):
        r, p, n = int(req[b]), int(start[b]), int(count[b])
        if not 0 <= r < bounds.shape[0] or p < 0 or n <= 0 or n > M or p + n > L:
            continue
        for u in range(p // T, (p + n - 1) // T + 1):
            lo, hi = max(p, u * T), min(p + n, (u + 1) * T)
            part = k[b, lo - p:hi - p].astype(np.float64)
            low = np.where(np.isnan(part), np.inf, part).min(axis=0)
            high = np.where(np.isnan(part), -np.inf, part).max(axis=0)
            if lo > u * T:
                low = np.fmin(low, bounds[r, u, :, 0])
                high = np.fmax(high, bounds[r, u, :, 1])
            bounds[r, u, :, 0], bounds[r, u, :, 1] = low, high


def scores(q, bounds, req, seq_lens, T, L):
    """[B, S, NB], -inf past the sequence, and the sums of the terms' magnitudes."""
    B, S, Hq, D = q.shape
    R, NB, H = bounds.shape[:3]
    out = np.full((B, S, NB), -np.inf)
    size = np.zeros((B, S, NB))
    for b in range(B):
        n = min(int(seq_lens[b]), L) if 0 <= req[b] < R else 0
        nb = max(0, -(-n // T))
        x = bounds[req[b], :nb] if nb else None
        for s in range(S):
            if nb:
                low = x[:, :, 0].repeat(Hq // H, axis=1) * q[b, s]
                high = x[:, :, 1].repeat(Hq // H, axis=1) * q[b, s]
                out[b, s, :nb] = np.maximum(low, high).sum(axis=(1, 2))
                size[b, s, :nb] = np.maximum(abs(low), abs(high)).sum(axis=(1, 2))
    return out, size


def select(score, seq_lens, req, R, T, L, n_select, first, last):
    """blocks [B, S, n_select] and their tokens, from scores in 64 bits."""
    B, S, _ = score.shape
    blocks = np.full((B, S, n_select), -1, np.int64)
    topk = np.full((B, S, n_select * T), -1, np.int64)
    for b in range(B):
        n = max(0, min(int(seq_lens[b]), L)) if 0 <= req[b] < R else 0
        nb = -(-n // T)
        for s in range(S):
            if nb <= n_select:
                got = np.arange(nb)
            else:
                open_ = np.arange(first, nb - last)
                z = score[b, s, open_]
                order = open_[np.lexsort((open_, -np.where(np.isnan(z), -np.inf, z), np.isnan(z)))]
                k = n_select - first - last
                got = np.sort(np.concatenate((np.arange(first), order[:k], np.arange(nb - last, nb))))
            blocks[b, s, :len(got)] = got
            t = (got[:, None] * T + np.arange(T)).reshape(-1)
            topk[b, s, :len(t)] = np.where(t < n, t, -1)
    return blocks, topk


def attend(q, rows, scales, prefix, lens, starts, T, heads, code, sm_scale, join=None):
    """out, lse and what error bounds are made of.  rows [R, L, W], scales [R, NB, 2, heads]."""
    B, S, Hq, D = q.shape
    R, L = rows.shape[:2]
    G = Hq // heads
    out, spread, biggest = (np.zeros((B, S, Hq, D)) for _ in range(3))
    lse, logit = np.full((B, S, Hq), -np.inf), np.zeros((B, S, Hq))
    taken = 0
    for g in range(len(prefix)):
        lo = max(min(max(int(starts[g]), 0), B), taken)
        hi = max(min(max(int(starts[g + 1]), 0), B), lo)
        taken = hi
        n = min(max(int(lens[g]), 0), L)
        if not 0 <= prefix[g] < R or n == 0 or hi == lo:
            continue
        x = ref.unpack(rows[prefix[g], :n], heads, D, code)
        x = x * scales[prefix[g], np.arange(n) // T].astype(np.float64)[..., None]
        for i in range(Hq):
            k, v = x[:, 0, i // G], x[:, 1, i // G]
            z = q[lo:hi, :, i] @ k.T * sm_scale
            logit[lo:hi, :, i] = (np.abs(q[lo:hi, :, i]) @ np.abs(k).T).max(axis=-1) * abs(sm_scale)
            top = z.max(axis=-1, keepdims=True)
            top = np.where(np.isfinite(top), top, 0)
            lse[lo:hi, :, i] = (top + np.log(np.exp(z - top).sum(axis=-1, keepdims=True)))[..., 0]
            p = np.exp(z - lse[lo:hi, :, i][..., None])
            out[lo:hi, :, i] = p @ v
            spread[lo:hi, :, i] = p @ np.abs(v)
            biggest[lo:hi, :, i] = np.abs(v).max(axis=0)
    if join is not None:
        other, other_lse = join
        both = np.logaddexp(lse, other_lse)
        safe = np.where(np.isneginf(both), 0, both)
        a, b = np.exp(lse - safe)[..., None], np.exp(other_lse - safe)[..., None]
        out = a * out + np.where(b > 0, b * other, 0)
        spread, biggest = a * spread + np.where(b > 0, b * np.abs(other), 0), a * biggest
        lse = both
    return {"out": out, "lse": lse, "spread": spread, "logit": logit, "biggest": biggest}


def frequencies(rot, base=10000.0):
    return [base ** (-2 * j / rot) for j in range(rot // 2)]
