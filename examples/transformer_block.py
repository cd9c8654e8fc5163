#!/usr/bin/env python3
"""The attention half of a diffusion transformer block on MXFP4 weights, every
step of it in this package's kernels:

    vec -> quantize_mxfp4_act -> gemm_mxfp4_few            shift, scale, gate
    x   -> block_norm (layer norm, scale, shift) -> quantize_mxfp4_act -> gemm_mxfp4   q, k, v
    q, k -> rotary_axes (time, height, width), in place
    q -> cross_attention to the image's keys, and to a text encoder's states
         (a length per sequence), joined by their log-sum-exps
    -> quantize_mxfp4_act -> gemm_mxfp4 -> block_norm (gate, residual, the other half's norm)

    python examples/transformer_block.py [--height 64 --width 64 --text 512 --heads 24 --batch 1]

Prints the time of a pass and how far the result is from the same block in
elementary torch operations in float32 (weights and activations of the layers
rounded to the same 4-bit values).
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_quantized_gemm_amd as w4  # noqa: E402

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def dequantize(codes, scales):
    """MXFP4 codes [rows, K/2] and scales [K/32, rows] -> float32 [rows, K]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = table[torch.stack([codes & 15, codes >> 4], -1).flatten(1).long()]
    return (v.unflatten(1, (-1, 32)) * torch.exp2(scales.t().float() - 127)[..., None]).flatten(1)


def rounded(x):
    """x at MXFP4's values: blocks of 32, scale 2^(floor(log2 max) - 2), nearest E2M1 value, ties to the even code."""
    v = x.to(torch.bfloat16).float().unflatten(-1, (-1, 32))
    scale = torch.exp2(torch.floor(torch.log2(v.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -100))) - 2)
    a = v.abs() / scale
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.sign(v) * (torch.round(a / step) * step).clamp(max=6.0) * scale).flatten(-2)


class Linear:
    """y = x W^T + bias + (x down^T) up with W held in MXFP4."""

    def __init__(self, n_in, n_out, rank, gen, device):
        def normal(*shape, std):
            return (torch.randn(shape, generator=gen, device=device) * std).to(torch.bfloat16)
        self.wgt, self.wscales, _ = w4.quantize_mxfp4_act(normal(n_out, n_in, std=n_in ** -0.5))
        self.one = torch.ones(n_out, device=device)
        self.bias = torch.zeros(n_out, device=device)
        self.down, self.up = normal(rank, n_in, std=n_in ** -0.5), normal(rank, n_out, std=0.1)

    def __call__(self, x):
        act, scales, low = w4.quantize_mxfp4_act(x, self.down)
        product = w4.gemm_mxfp4_few if x.shape[0] <= w4.FEW_MAX_M else w4.gemm_mxfp4
        return product(act, scales, self.wgt, self.wscales, self.one, self.bias, low, self.up)

    def plain(self, x):
        return rounded(x) @ dequantize(self.wgt, self.wscales).t() + (x @ self.down.float().t()) @ self.up.float()


class Block:
    def __init__(self, heads, head_dim=128, rank=32, sections=None, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.heads, self.dim = heads, head_dim
        hidden = heads * head_dim
        self.modulation = Linear(hidden, 3 * hidden, rank, gen, device)
        self.qkv = Linear(hidden, 3 * hidden, rank, gen, device)
        self.text_kv = Linear(hidden, 2 * hidden, rank, gen, device)
        self.out = Linear(hidden, hidden, rank, gen, device)
        half = head_dim // 2
        self.sections = sections or (half - 2 * (half * 7 // 16), half * 7 // 16, half * 7 // 16)
        self.inv_freq = torch.cat([10000.0 ** (-torch.arange(n, device=device, dtype=torch.float64) / n)
                                   for n in self.sections]).float()

    def __call__(self, x, vec, text, text_lens, positions):
        """x [B, L, hidden], vec [B, hidden], text [B, T, hidden] bfloat16; text_lens
        int32 [B]; positions int32 [L, 3] -> [B, L, hidden]."""
        B, L, hidden = x.shape
        H, D = self.heads, self.dim
        shift, scale, gate = self.modulation(vec)[:, None].chunk(3, -1)
        h, _ = w4.block_norm(x, scale=scale, shift=shift, eps=1e-5)
        joint = self.qkv(h.reshape(B * L, hidden)).view(B, L, 3 * H, D)
        turned = joint[:, :, :2 * H]
        w4.rotary_axes(turned, positions, self.inv_freq, self.sections, out=turned)
        q, k, v = joint[:, :, :H], joint[:, :, H:2 * H], joint[:, :, 2 * H:]
        states = self.text_kv(text.reshape(-1, hidden)).view(B, -1, 2 * H, D)
        image, li = w4.cross_attention(q, k, v, return_lse=True)
        words, lw = w4.cross_attention(q, states[:, :, :H], states[:, :, H:], kv_lens=text_lens, return_lse=True)
        share = torch.sigmoid(lw - li).transpose(1, 2)[..., None]      # the words' part of all weights
        o = torch.lerp(image.float(), words.float(), share).to(x.dtype)
        # (with it comes the norm that the block's other half begins with)
        return w4.block_norm(x, self.out(o.view(B * L, hidden)).view(B, L, hidden), gate=gate, eps=1e-5)[1]

    def plain(self, x, vec, text, text_lens, positions):
        x, vec, text = x.float(), vec.float(), text.float()
        B, L, hidden = x.shape
        H, D = self.heads, self.dim
        shift, scale, gate = self.modulation.plain(vec)[:, None].chunk(3, -1)
        h = torch.nn.functional.layer_norm(x, (hidden,)) * (1 + scale) + shift
        q, k, v = self.qkv.plain(h).view(B, L, 3 * H, D).split(H, 2)
        axis = torch.repeat_interleave(torch.arange(3), torch.tensor(self.sections)).to(x.device)
        t = (positions.float()[:, axis] * self.inv_freq)[:, None]
        turn = torch.polar(torch.ones_like(t), t)
        q, k = (torch.view_as_real(torch.view_as_complex(a.reshape(B, L, H, D // 2, 2)) * turn).flatten(-2) for a in (q, k))
        kt, vt = self.text_kv.plain(text).view(B, -1, 2 * H, D).split(H, 2)
        k, v = torch.cat([k, kt], 1), torch.cat([v, vt], 1)
        s = (q.transpose(1, 2) @ k.permute(0, 2, 3, 1).contiguous()) * D ** -0.5
        dead = torch.arange(text.shape[1], device=x.device) >= text_lens[:, None]
        s[..., L:].masked_fill_(dead[:, None, None], float("-inf"))
        o = torch.softmax(s, -1) @ v.transpose(1, 2).contiguous()
        return x + gate * self.out.plain(o.transpose(1, 2).reshape(B, L, hidden))


def inputs(batch, height, width, text, hidden, seed=1, device="cuda"):
    gen = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=device).to(torch.bfloat16)
    at = torch.arange(height * width, device=device)
    positions = torch.stack([torch.zeros_like(at), at // width, at % width], -1).to(torch.int32)
    lens = torch.tensor([max(0, text - b * (text // 3)) for b in range(batch)], dtype=torch.int32, device=device)
    return normal(batch, height * width, hidden), normal(batch, hidden), normal(batch, text, hidden), lens, positions


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("height", 64), ("width", 64), ("text", 512), ("heads", 24), ("batch", 1), ("steps", 20)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args(argv)
    block = Block(a.heads)
    args = inputs(a.batch, a.height, a.width, a.text, a.heads * block.dim)
    y = block(*args)
    want = block.plain(*args)
    change = want - args[0].float()
    far = ((y.float() - want).norm() / change.norm()).item()
    torch.cuda.synchronize()
    begin = time.perf_counter()
    for _ in range(a.steps):
        block(*args)
    torch.cuda.synchronize()
    ms = (time.perf_counter() - begin) / a.steps * 1e3
    print(f"{a.batch} x {a.height * a.width} tokens, {a.text} text states, {a.heads} heads: {ms:.3f} ms a pass; "
          f"differs from the plain block by {far:.3f} of what the block adds", flush=True)
    return far


if __name__ == "__main__":
    main()
