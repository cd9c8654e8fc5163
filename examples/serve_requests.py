#!/usr/bin/env python3
"""The attention half of a decoder block on MXFP4 weights, serving several requests
at once, each with a low-rank adapter of its own:

    x -> block_norm -> quantize_mxfp4_act -> gemm_mxfp4 -> lora_adapters    q, k, v
    q, k -> rotary_axes, in place;   k, v -> cache_append
    prompts of different lengths, packed:  packed_attention
    then one new token of each request:    paged_attention over the cache
    -> quantize_mxfp4_act -> gemm_mxfp4 (few rows: gemm_mxfp4_few) -> lora_adapters
    -> block_norm: norm of the result, residual, norm of the block's other half

    python examples/serve_requests.py [--prompts 700,300,41,1 --tokens 8 --heads 24 --kv-heads 8]

Prints the time of the prompts' pass and of a token's, and how far both are
from the same block in elementary torch operations in float32 over whole sequences (weights
and activations of the layers rounded to the same 4-bit values).
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import bit_quantized_gemm_amd as w4  # noqa: E402
from transformer_block import Linear  # noqa: E402


class Adapters:
    """Low-rank adapters of ranks of their own beside one projection."""

    def __init__(self, count, n_in, n_out, rank, gen, device):
        def normal(*shape, std):
            return (torch.randn(shape, generator=gen, device=device) * std).to(torch.bfloat16)
        self.down, self.up = normal(count, rank, n_in, std=n_in ** -0.5), normal(count, rank, n_out, std=0.2)
        self.ranks = torch.tensor([max(1, rank >> (a % 3)) for a in range(count)], dtype=torch.int32, device=device)
        self.scaling = torch.rand(count, generator=gen, device=device) + 0.5

    def add(self, y, x, which):
        """y += what each row's adapter gives for x; which int32 [rows], -1: none."""
        return w4.lora_adapters(y, x, self.down, self.up, which, scaling=self.scaling, ranks=self.ranks, out=y)

    def plain(self, x, a):
        r = int(self.ranks[a])
        return (x @ self.down[a, :r].float().t()) @ self.up[a, :r].float() * self.scaling[a]


class Cache:
    """Pages of keys and values, and each request's table of them."""

    def __init__(self, requests, most, kv_heads, head_dim, page, device):
        self.page, width = page, -(-most // page)
        self.k, self.v = torch.zeros(2, requests * width, page, kv_heads, head_dim, dtype=torch.bfloat16, device=device)
        self.table = torch.randperm(requests * width, device=device).to(torch.int32).view(requests, width)

    def slots(self, request, position):
        """Places of the tokens at `position` of `request` (int64 tensors)."""
        return self.table[request, position // self.page].long() * self.page + position % self.page


class Block:
    def __init__(self, heads, kv_heads, adapters, head_dim=128, rank=32, adapter_rank=16, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.heads, self.kv_heads, self.dim = heads, kv_heads, head_dim
        hidden, out = heads * head_dim, (heads + 2 * kv_heads) * head_dim
        self.qkv, self.out = Linear(hidden, out, rank, gen, device), Linear(hidden, hidden, rank, gen, device)
        self.qkv_adapters = Adapters(adapters, hidden, out, adapter_rank, gen, device)
        self.out_adapters = Adapters(adapters, hidden, hidden, adapter_rank, gen, device)
        self.before, self.after, self.other = (
            (1 + 0.1 * torch.randn(hidden, generator=gen, device=device)).to(torch.bfloat16) for _ in range(3))
        half = head_dim // 2
        self.inv_freq = (10000.0 ** (-torch.arange(half, device=device, dtype=torch.float64) / half)).float()

    def project(self, x, position, which, slots, cache):
        """q, k, v [tokens, heads, head_dim] of x [tokens, hidden], rotated; k and v go to the cache."""
        h, _ = w4.block_norm(x, kind="rms", weight=self.before)
        joint = self.qkv_adapters.add(self.qkv(h), h, which).view(1, len(x), -1, self.dim)
        turned = joint[:, :, :self.heads + self.kv_heads]
        w4.rotary_axes(turned, position.view(-1, 1).to(torch.int32), self.inv_freq, (self.dim // 2,), interleaved=False, out=turned)
        q, k, v = joint[0].split([self.heads, self.kv_heads, self.kv_heads], 1)
        w4.cache_append(k, v, cache.k, cache.v, slots)
        return q, k, v

    def finish(self, x, o, which):
        """(the other half's input, the residual stream) from the attention's result o."""
        o = o.reshape(x.shape)
        y = self.out_adapters.add(self.out(o), o, which)
        return w4.block_norm(x, y, post_norm=True, post_weight=self.after, kind="rms", weight=self.other)

    def prompts(self, x, lens, which, cache):
        """x [sum of lens, hidden], the prompts one after the other; which int32 [requests]: their adapters."""
        lens = torch.tensor(lens, device=x.device)
        ends = lens.cumsum(0)
        starts = torch.cat([ends.new_zeros(1), ends]).to(torch.int32)
        request = torch.repeat_interleave(torch.arange(len(lens), device=x.device), lens)
        position = torch.arange(len(x), device=x.device) - starts[request]
        which = which[request]
        q, k, v = self.project(x, position, which, cache.slots(request, position), cache)
        return self.finish(x, w4.packed_attention(q, k, v, starts), which)

    def tokens(self, x, lens, which, cache):
        """x [requests, hidden], one new token each; lens int32 [requests]: tokens before it."""
        request = torch.arange(len(x), device=x.device)
        q, _, _ = self.project(x, lens, which, cache.slots(request, lens.long()), cache)
        o = w4.paged_attention(q[:, None], cache.k, cache.v, cache.table, lens + 1)
        return self.finish(x, o, which)

    def plain(self, x, a):
        """Both results for one whole sequence x [tokens, hidden] of a request with adapter a (-1: none)."""
        def norm(v, w):
            return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + 1e-6) * w.float()

        def layer(linear, adapters, v):
            return linear.plain(v) + (adapters.plain(v, a) if a >= 0 else 0.0)
        x = x.float()
        n, H, G, D = len(x), self.heads, self.kv_heads, self.dim
        q, k, v = layer(self.qkv, self.qkv_adapters, norm(x, self.before)).view(n, -1, D).split([H, G, G], 1)
        t = torch.arange(n, device=x.device)[:, None, None] * self.inv_freq
        turn = torch.polar(torch.ones_like(t), t)
        q, k = (torch.view_as_real(torch.complex(*h.chunk(2, -1)) * turn).transpose(-1, -2).flatten(-2) for h in (q, k))
        k, v = (h.repeat_interleave(H // G, 1) for h in (k, v))
        s = (q.transpose(0, 1) @ k.permute(1, 2, 0).contiguous()) * D ** -0.5
        s.masked_fill_(torch.ones(n, n, dtype=torch.bool, device=x.device).triu(1), float("-inf"))
        o = (torch.softmax(s, -1) @ v.transpose(0, 1).contiguous()).transpose(0, 1).reshape(n, -1)
        r = x + norm(layer(self.out, self.out_adapters, o), self.after)
        return norm(r, self.other), r


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--prompts", default="700,300,41,1")
    for name, value in (("tokens", 8), ("heads", 24), ("kv-heads", 8), ("adapters", 3), ("page", 64), ("steps", 20)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args(argv)
    lens = [int(n) for n in a.prompts.split(",")]
    block = Block(a.heads, a.kv_heads, a.adapters)
    hidden, device = a.heads * block.dim, "cuda"
    gen = torch.Generator(device=device).manual_seed(1)
    seqs = [torch.randn(n + a.tokens, hidden, generator=gen, device=device).to(torch.bfloat16) for n in lens]
    adapters = [i % (a.adapters + 1) - 1 for i in range(len(lens))]       # the first request has none
    which = torch.tensor(adapters, dtype=torch.int32, device=device)
    cache = Cache(len(lens), max(lens) + a.tokens, a.kv_heads, block.dim, a.page, device)

    packed = torch.cat([s[:n] for s, n in zip(seqs, lens)])
    first = block.prompts(packed, lens, which, cache)
    before = torch.tensor(lens, dtype=torch.int32, device=device)
    steps = [block.tokens(torch.stack([s[n + i] for s, n in zip(seqs, lens)]), before + i, which, cache) for i in range(a.tokens)]
    off, size, at = [0.0, 0.0], [0.0, 0.0], 0
    for b, (s, n) in enumerate(zip(seqs, lens)):
        want = block.plain(s, adapters[b])
        for j, (w, begin) in enumerate(zip(want, (torch.zeros_like(s), s))):     # of the residual: what the block adds
            got = torch.cat([first[j][at:at + n]] + [t[j][b:b + 1] for t in steps]).float()
            off[j] += (got - w).square().sum().item()
            size[j] += (w - begin.float()).square().sum().item()
        at += n
    far = max((o / z) ** 0.5 for o, z in zip(off, size))

    def timed(f):
        torch.cuda.synchronize()
        begin = time.perf_counter()
        for _ in range(a.steps):
            f()
        torch.cuda.synchronize()
        return (time.perf_counter() - begin) / a.steps * 1e3
    now = torch.stack([s[n] for s, n in zip(seqs, lens)])
    print(f"{len(lens)} requests, {sum(lens)} tokens: prompts {timed(lambda: block.prompts(packed, lens, which, cache)):.3f} ms, "
          f"a token of each {timed(lambda: block.tokens(now, before, which, cache)):.3f} ms; differs from the plain block by "
          f"{far:.3f} of what the block adds", flush=True)
    return far


if __name__ == "__main__":
    main()
