"""Decoding over a host-resident 8-bit key/value cache whose tokens are selected by bounds on
their keys, behind a prompt that all requests share: every step normalises and turns the new
queries and keys, appends them, brings the keys into their blocks' bounds, selects blocks,
swaps their rows in, attends over them and joins the attention over the shared prompt, which
stays in device memory once for all.

    python examples/decode_selected.py [--requests 32] [--steps 100]

Inputs are random.  Prints the time of a step and how much of the attention's weight over
the requests' own tokens the selected blocks held in the last one.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import sparse_attention_kv_swap_gb300 as hs  # noqa: E402
from sparse_attention_kv_swap_gb300.cache import SwapInCache  # noqa: E402


class SelectingDecoder:
    """One attention layer of `requests` sequences of up to `limit` tokens behind a shared prompt."""

    def __init__(self, requests, limit, shared, blocks, kv_heads=8, group=4, head_dim=128,
                 block_tokens=64, code=hs.HS_KV_E4M3, dtype=torch.bfloat16, base=10000.0):
        self.fmt = hs.make_kv_format(kv_heads, head_dim, block_tokens, code)
        self.T, self.shared, self.dim, self.dtype = block_tokens, shared, head_dim, dtype
        self.heads, self.requests = kv_heads * group, requests
        top_k = blocks * block_tokens
        self.cache = SwapInCache(hs.make_config(requests, limit, self.fmt.item_size_bytes, 2 * top_k,
                                                top_k, 1, extra_page_size=block_tokens))
        self.scales = self.cache.kv_scales(self.fmt)
        self.bounds = self.cache.key_bounds(self.fmt, dtype, block_tokens)
        self.rope = hs.make_rope([base ** (-2 * j / head_dim) for j in range(head_dim // 2)])
        self.weight = [torch.ones(head_dim, device="cuda") for _ in range(2)]  # queries, keys
        i32 = dict(dtype=torch.int32, device="cuda")
        self.req = torch.arange(requests, **i32)
        self.one = torch.ones(requests, **i32)
        self.lens = torch.zeros(requests, **i32)
        self.rows = torch.empty((1, shared, self.fmt.item_size_bytes), dtype=torch.uint8,
                                device="cuda")
        self.shared_scales = torch.zeros(self.fmt.scales_shape(1, shared), device="cuda")
        self.prefix = torch.zeros(1, **i32)
        self.prefix_len = torch.tensor([shared], **i32)
        self.starts = torch.tensor([0, requests], **i32)
        self.selected, self.own, self.out = {}, {}, {}

    def _turn(self, q, k, first):
        """New queries and keys at positions first[b], first[b] + 1, ...: normalised and turned."""
        at = first[:, None] + torch.arange(k.shape[1], dtype=torch.int32, device="cuda")
        q_out, k_out = None if q is None else torch.empty_like(q), torch.empty_like(k)
        hs.hs_norm_rope(q, k, at, self.rope, q_out, k_out, self.weight[0], self.weight[1])
        return q_out, k_out

    def share(self, k, v):
        """The prompt of all: k, v [1, shared, kv_heads, head_dim]."""
        k = self._turn(None, k, self.prefix)[1]
        hs.hs_quantize_kv(self.fmt, k, v, self.prefix, self.prefix, self.prefix_len, self.rows,
                          self.shared_scales)
        return k

    def append(self, k, v, count):
        """Own tokens of the requests, normalised and turned: [requests, tokens, kv_heads, head_dim],
        the first count[b] of them."""
        self.cache.append_kv(self.fmt, self.scales, k, v, self.req, self.lens, count)
        self.cache.bound_keys(self.bounds, self.T, k, self.req, self.lens, count)
        self.lens += count

    def prompt(self, k, v, count):
        """The requests' own prompts, before norm and rotation."""
        k = self._turn(None, k, self.lens + self.shared)[1]
        self.append(k, v, count)
        return k

    def step(self, q, k, v):
        """One token: q [requests, 1, heads, head_dim], k and v [requests, 1, kv_heads, head_dim]."""
        self.q, self.k = self._turn(q, k, self.lens + self.shared)
        self.append(self.k, v, self.one)
        self.selected.update(self.cache.select_blocks(self.bounds, self.T, self.q, self.req,
                                                      self.lens, out=self.selected))
        topk = self.selected["topk"]
        self.selected.update(self.cache.swap_in(self.req, self.lens, topk, out=self.selected))
        self.own.update(self.cache.attend(self.fmt, self.scales, self.q, topk,
                                          self.selected["device_locs"], self.req, lse=True,
                                          out=self.own))
        self.out.update(self.cache.attend_prefix(self.fmt, self.rows, self.shared_scales, self.q,
                                                 self.prefix, self.prefix_len, self.starts,
                                                 join=self.own, out=self.out))
        return self.out["out"]


def main():
    p = argparse.ArgumentParser(description=__doc__,
                                formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--requests", type=int, default=32)
    p.add_argument("--steps", type=int, default=100)
    p.add_argument("--limit", type=int, default=8192)
    p.add_argument("--shared", type=int, default=8192)
    p.add_argument("--blocks", type=int, default=16)
    a = p.parse_args()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    d = SelectingDecoder(a.requests, a.limit, a.shared, a.blocks)
    kv = d.fmt.num_kv_heads

    def rand(*shape):
        return torch.randn(shape, device="cuda", generator=gen).to(d.dtype)

    d.share(rand(1, a.shared, kv, d.dim), rand(1, a.shared, kv, d.dim))
    n = a.limit - a.steps
    k, v = rand(a.requests, n, kv, d.dim), rand(a.requests, n, kv, d.dim)
    keys = [d.prompt(k, v, torch.full_like(d.lens, n))]

    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for i in range(a.steps):
        q, k, v = rand(a.requests, 1, d.heads, d.dim), rand(a.requests, 1, kv, d.dim), rand(
            a.requests, 1, kv, d.dim)
        if i == 1:
            begin.record()
        d.step(q, k, v)
        keys.append(d.k)
    end.record()
    end.synchronize()
    k = torch.cat(keys, 1)[:1].float().repeat_interleave(d.heads // kv, 2)
    w = torch.softmax(torch.einsum("bhd,bkhd->bhk", d.q[:1, 0].float(), k) * d.dim ** -0.5, 2)
    at = d.selected["topk"][0, 0].long()
    held = w[0, :, at[at >= 0]].sum(1).mean().item()
    rc, flags = d.cache.status()
    assert rc == 0 and flags == 0
    if a.steps > 1:
        print("%d requests of %d tokens behind %d shared ones: %.0f us a step" % (
            a.requests, a.limit, a.shared, begin.elapsed_time(end) * 1e3 / (a.steps - 1)))
    print("%d of %d blocks held %.1f%% of the weight" % (
        a.blocks, -(-a.limit // d.T), 100 * held))
    d.cache.close()


if __name__ == "__main__":
    main()
