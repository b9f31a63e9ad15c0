"""Decoding with an 8-bit key/value cache that is kept in host memory: a prompt is quantised
and written back, every step appends the new tokens' keys and values, swaps in the selected
rows, attends over them and adds up their attention weights, and a sequence that reaches
`limit` tokens is cut to the `budget` that got most weight.

    python examples/decode_8bit.py [--requests 8] [--steps 200]

Inputs are random; the selection that a model's indexer would make is the newest token and a
random choice.  Prints the time of a step and the error that 8-bit rows make.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import sparse_attention_kv_swap_gb300 as hs  # noqa: E402
from sparse_attention_kv_swap_gb300.cache import SwapInCache  # noqa: E402


class Decoder:
    """One attention layer's cache of `requests` sequences."""

    def __init__(self, requests, limit, budget, recent, top_k, hot, kv_heads=8, group=4,
                 head_dim=128, block_tokens=64, code=hs.HS_KV_E4M3, dtype=torch.bfloat16):
        self.fmt = hs.make_kv_format(kv_heads, head_dim, block_tokens, code)
        self.limit, self.budget, self.recent, self.top_k = limit, budget, recent, top_k
        cfg = hs.make_config(requests, limit, self.fmt.item_size_bytes, hot, top_k, 1,
                             extra_page_size=block_tokens)
        self.cache = SwapInCache(cfg)
        self.scales = self.cache.kv_scales(self.fmt)
        self.acc = torch.zeros((requests, limit), device="cuda")
        self.req = torch.arange(requests, dtype=torch.int32, device="cuda")
        self.lens = [0] * requests
        self.seq_lens = torch.zeros(requests, dtype=torch.int32, device="cuda")
        self.heads, self.dim, self.dtype = kv_heads * group, head_dim, dtype
        self.out = {}

    def prompt(self, k, v, lens):
        """k, v [requests, tokens, kv_heads, head_dim]; request i has the first lens[i] tokens."""
        self.lens = list(lens)
        self.seq_lens.copy_(torch.tensor(self.lens, dtype=torch.int32))
        self.cache.append_kv(self.fmt, self.scales, k, v, self.req,
                             torch.zeros_like(self.seq_lens), self.seq_lens)

    def make_room(self):
        """Cuts the sequences that have reached the limit; returns them."""
        full = [i for i, n in enumerate(self.lens) if n == self.limit]
        if full:
            kept = self.cache.evict(self.fmt, [self.scales], [self.acc], full,
                                    [self.limit] * len(full), self.budget, self.recent)
            for i, n in zip(full, kept):
                self.lens[i] = n
            self.seq_lens.copy_(torch.tensor(self.lens, dtype=torch.int32))
        return full

    def step(self, q, k, v, topk):
        """One token: q [requests, 1, heads, head_dim], k and v [requests, 1, kv_heads, head_dim],
        topk [requests, 1, top_k] (-1 where a sequence is shorter)."""
        self.cache.append_kv(self.fmt, self.scales, k, v, self.req, self.seq_lens,
                             torch.ones_like(self.seq_lens))
        self.seq_lens += 1
        self.lens = [n + 1 for n in self.lens]
        self.out.update(self.cache.swap_in(self.req, self.seq_lens, topk, out=self.out))
        self.out.update(self.cache.attend(self.fmt, self.scales, q, topk,
                                          self.out["device_locs"], self.req, lse=True,
                                          weights=True, acc=self.acc, out=self.out))
        return self.out["out"]

    def select(self, generator=None):
        """The newest token and a random choice of the others."""
        draw = torch.rand((len(self.lens), self.limit), device="cuda", generator=generator)
        n = self.seq_lens.long()[:, None] + 1  # with the token that the step appends
        at = torch.arange(self.limit, device="cuda")
        draw = draw.masked_fill(at >= n, -1.0).masked_fill(at == n - 1, 2.0)
        value, topk = draw.topk(min(self.top_k, self.limit), dim=1)
        topk = torch.nn.functional.pad(topk.masked_fill(value < 0, -1),
                                       (0, self.top_k - topk.shape[1]), value=-1)
        return topk.to(torch.int32)[:, None].contiguous()


def main():
    p = argparse.ArgumentParser(description=__doc__,
                                formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--requests", type=int, default=8)
    p.add_argument("--steps", type=int, default=200)
    p.add_argument("--limit", type=int, default=4096)
    p.add_argument("--top-k", type=int, default=1024)
    a = p.parse_args()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    d = Decoder(a.requests, a.limit, a.limit // 2, a.limit // 16, a.top_k, 2 * a.top_k)

    def rand(*shape):
        return torch.randn(shape, device="cuda", generator=gen).to(d.dtype)

    kv = d.fmt.num_kv_heads
    n = a.limit - a.steps // 2
    k, v = rand(a.requests, n, kv, d.dim), rand(a.requests, n, kv, d.dim)
    d.prompt(k, v, [n] * a.requests)

    # What 8 bits cost: one step over the prompt, against attention on the values before.
    q, k1, v1, topk = rand(a.requests, 1, d.heads, d.dim), rand(a.requests, 1, kv, d.dim), rand(
        a.requests, 1, kv, d.dim), d.select(gen)
    out = d.step(q, k1, v1, topk).float()
    at = topk.long()[:, 0, :, None, None].expand(-1, -1, kv, d.dim)
    ks = torch.cat([k, k1], 1).gather(1, at).float().repeat_interleave(d.heads // kv, 2)
    vs = torch.cat([v, v1], 1).gather(1, at).float().repeat_interleave(d.heads // kv, 2)
    w = torch.softmax(torch.einsum("bhd,bkhd->bhk", q[:, 0].float(), ks) * d.dim ** -0.5, 2)
    want = torch.einsum("bhk,bkhd->bhd", w, vs)[:, None]
    print("error of the 8-bit rows: %.4f of the output's size"
          % ((out - want).norm() / want.norm()).item())

    cut, begin, end = 0, torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(a.steps - 1):
        cut += len(d.make_room())
        d.step(rand(a.requests, 1, d.heads, d.dim), rand(a.requests, 1, kv, d.dim),
               rand(a.requests, 1, kv, d.dim), d.select(gen))
    end.record()
    end.synchronize()
    rc, flags = d.cache.status()
    assert rc == 0 and flags == 0
    print("%d steps of %d requests, %d sequences cut to %d tokens: %.0f us a step"
          % (a.steps - 1, a.requests, cut, d.budget, begin.elapsed_time(end) * 1e3 / (a.steps - 1)))
    d.cache.close()


if __name__ == "__main__":
    main()
