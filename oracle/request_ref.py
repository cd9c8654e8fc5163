"""Plain CPU oracles of the operators that serve many requests at once, in
float64, each with the error bound its kernel is held to.

TEST INFRASTRUCTURE ONLY. The product (``bit_quantized_gemm_amd``) never
imports it and shares no code with it.

Tensors come as float64 arrays of the 16-bit inputs' values, with dtype "bf16"
or "f16".
"""
from __future__ import annotations

import numpy as np

from .block_ref import half_spacing

__all__ = ["block_norm_ref", "cache_append_ref", "lora_adapters_ref", "packed_attention_ref", "paged_attention_ref"]

# relative error of a float32 sum of a row: at most 64 additions in a lane and 12
# across lanes and waves, each off by 2^-24 of the partial sum
SUM = 76 * 2.0 ** -24


def _norm(v, layer, eps, err):
    """norm(v), and how far the kernel's may be off when its v is off by at most err."""
    mean = v.mean(-1, keepdims=True) if layer else 0.0
    d = v - mean
    rstd = 1.0 / np.sqrt((d * d).mean(-1, keepdims=True) + eps)
    n = d * rstd
    size = np.abs(v).mean(-1, keepdims=True)
    # of the mean: SUM of the mean magnitude, and v's own error; the difference and the
    # product round once each (2^-24), the square root and the division within 2^-21 together
    of_mean = (SUM * size + err.mean(-1, keepdims=True)) if layer else 0.0
    of_d = of_mean + err + 2.0 ** -23 * np.abs(v)
    # of 1 / sqrt(var + eps), relative: half of the sum's, of the common shift's and of v's
    rms = np.sqrt((of_d * of_d).mean(-1, keepdims=True))
    of_rstd = SUM + rms * rstd + 2.0 ** -21
    return n, rstd * of_d * (1 + of_rstd) + np.abs(n) * of_rstd


def block_norm_ref(x, y=None, gate=None, residual_scale=1.0, post_norm=False, post_weight=None, layer=True, weight=None,
                   bias=None, scale=None, shift=None, eps=1e-6, dtype="bf16"):
    """x, y [..., width], the others broadcast to it -> (out, residual, bounds of both)."""
    u = 2.0 ** -24
    one = np.ones_like(x)
    r, err = x.copy(), np.zeros_like(x)
    if y is not None:
        z, ez = y.copy(), np.zeros_like(x)
        if post_norm:
            z, ez = _norm(y, layer, eps, ez)
            w = one if post_weight is None else post_weight
            z, ez = z * w, ez * np.abs(w) + 2 * u * np.abs(z * w)
        g = one if gate is None else gate
        z, ez = z * g, ez * np.abs(g) + 2 * u * np.abs(z * g)
        a = float(np.float32(residual_scale))
        r = a * x + z
        err = ez + 2 * u * (np.abs(a * x) + np.abs(z))
    n, en = _norm(r, layer, eps, err)
    for factor, term in ((weight, bias), (None if scale is None else 1 + scale, shift)):
        f = one if factor is None else factor
        t = 0.0 if term is None else term
        # (1 + scale is not rounded by itself: n + n scale, two roundings)
        en = en * np.abs(f) + 4 * u * (np.abs(n) * (1 + np.abs(f)) + np.abs(t))
        n = n * f + t
    return n, r, en + 0.5 * half_spacing(n, dtype) * (1 + 2.0 ** -6), err + 0.5 * half_spacing(r, dtype) * (1 + 2.0 ** -6)


def cache_append_ref(k, v, k_cache, v_cache, slots):
    """The caches [pages, page_size, heads, head_dim] after the tokens k, v [tokens, heads, head_dim] (any dtype)."""
    kc, vc = k_cache.copy(), v_cache.copy()
    pages, page = kc.shape[:2]
    for t, s in enumerate(slots):
        if 0 <= s < pages * page:
            kc[s // page, s % page] = k[t]
            vc[s // page, s % page] = v[t]
    return kc, vc


def lora_adapters_ref(y, x, down, up, adapter, scaling=None, ranks=None, dtype="bf16"):
    """y [rows, N], x [rows, K], down [A, R, K], up [A, R, N], adapter [rows] -> (out, bound).

    The bound, with L = |x| |down|^T, T = scaling L |up| and K-term float32 sums in an order
    of their own (products of 16-bit values are exact; a chain of at most K / 8 + 64
    additions, each off by 2^-24 of at most L): low off by (K / 8 + 64) 2^-24 L; its two 16-bit
    parts by 2^-17 (bf16: 2^-9 of 2^-9, and their products' rounding; f16 less), and,
    f16 after scaling to 2^15, by 2^-25 2^-14 of the largest low of the row for each part of
    it that is subnormal; the second sum by (R / 8 + 8) 2^-24 T."""
    rows, K = x.shape
    R = down.shape[1]
    out, bound = y.copy(), np.zeros_like(y)
    for m in range(rows):
        a = int(adapter[m])
        if not 0 <= a < down.shape[0]:
            continue
        r = R if ranks is None else min(max(int(ranks[a]), 0), R)
        s = 1.0 if scaling is None else float(np.float32(scaling[a]))
        d, w = down[a, :r], up[a, :r]
        low = d @ x[m]
        mag = np.abs(d) @ np.abs(x[m])
        out[m] += s * (low @ w)
        T = abs(s) * (mag @ np.abs(w))
        top = abs(s) * (np.abs(low).max() if r else 0.0)
        bound[m] = T * ((K / 8 + 64 + R / 8 + 8) * 2.0 ** -24) + abs(s) * (np.abs(low) @ np.abs(w)) * 2.0 ** -17 + \
            (2.0 ** -38 * top * np.abs(w).sum(0) if dtype == "f16" else 0.0) + 2.0 ** -23 * (np.abs(y[m]) + T)
    some = bound > 0
    return out, np.where(some, bound + 0.5 * half_spacing(out, dtype) * (1 + 2.0 ** -6), 0.0)


def _attend(q, k, v, sees, scale, dtype):
    """One head: q [n, D], k, v [m, D], sees [n]: row i sees the first sees[i] keys -> out, lse and their bounds.

    The bounds are those of attention_ref in block_ref.py: weights off by the unit
    roundoff of the 16-bit type and by twice the float32 error of their scores."""
    n, D = q.shape
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
    out, bound = np.zeros((n, D)), np.zeros((n, D))
    lse, lse_bound = np.full(n, -np.inf), np.zeros(n)
    m = int(max(sees.max(initial=0), 0))
    live = np.arange(m)[None, :] < sees[:, None]
    rows = live.any(1)
    if not rows.any():
        return out, lse, bound, lse_bound
    q, live = q[rows], live[rows]
    k, v = k[:m], v[:m]
    s = np.where(live, scale * (q @ k.T), -np.inf)
    top = s.max(axis=1, keepdims=True)
    p = np.exp(s - top)
    total = p.sum(axis=1, keepdims=True)
    o = p @ v / total
    ds = (D + 8) * 2.0 ** -24 * np.where(live, scale * (np.abs(q) @ np.abs(k).T), 0.0).max(axis=1, keepdims=True) \
        + 2.0 ** -22 * np.abs(np.where(live, s, 0.0)).max(axis=1, keepdims=True)
    T = p @ np.abs(v) / total
    tiny = 2.0 ** -25 * (live @ np.abs(v)) if dtype == "f16" else 0.0
    out[rows] = o
    lse[rows] = (top + np.log(total))[:, 0]
    bound[rows] = 2 * T * (u + 2 * ds + 2.0 ** -20) + 0.5 * half_spacing(o, dtype) * (1 + 2.0 ** -6) + tiny
    lse_bound[rows] = (2 * ds)[:, 0] + 2.0 ** -20 * (1 + np.abs(lse[rows]))
    return out, lse, bound, lse_bound


def packed_attention_ref(q, k, v, starts, causal=True, scale=None, dtype="bf16"):
    """q [T, HQ, D], k, v [T, HKV, D] -> (out, lse [HQ, T], their bounds, whether a token is in a sequence [T])."""
    T, HQ, D = q.shape
    group = HQ // k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    out, bound = np.zeros((T, HQ, D)), np.zeros((T, HQ, D))
    lse, lse_bound = np.full((HQ, T), -np.inf), np.zeros((HQ, T))
    inside = np.zeros(T, dtype=bool)
    at = np.clip(np.asarray(starts, dtype=np.int64), 0, T)
    for a, b in zip(at[:-1], at[1:]):
        n = b - a
        if n <= 0:
            continue
        inside[a:b] = True
        sees = np.arange(1, n + 1) if causal else np.full(n, n)
        for h in range(HQ):
            g = h // group
            out[a:b, h], lse[h, a:b], bound[a:b, h], lse_bound[h, a:b] = _attend(q[a:b, h], k[a:b, g], v[a:b, g], sees, scale, dtype)
    return out, lse, bound, lse_bound, inside


def paged_attention_ref(q, k_cache, v_cache, table, lens, scale=None, dtype="bf16"):
    """q [B, Q, HQ, D], caches [pages, page, HKV, D] -> (out, lse [B, HQ, Q], their bounds)."""
    B, Q, HQ, D = q.shape
    pages, page, HKV, _ = k_cache.shape
    group = HQ // HKV
    scale = D ** -0.5 if scale is None else scale
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    lse, lse_bound = np.full((B, HQ, Q), -np.inf), np.zeros((B, HQ, Q))
    for b in range(B):
        n = min(max(int(lens[b]), 0), table.shape[1] * page)
        keys = np.array([(table[b][j // page], j % page) for j in range(n)], dtype=np.int64).reshape(-1, 2)
        there = (keys[:, 0] >= 0) & (keys[:, 0] < pages)
        # keys of a page that is none are left out: of those that are, row i sees so many
        sees = np.array([int(there[:max(0, n - Q + 1 + i)].sum()) for i in range(Q)])
        keys = keys[there]
        for h in range(HQ):
            k, v = (c[keys[:, 0], keys[:, 1], h // group] for c in (k_cache, v_cache))
            out[b, :, h], lse[b, h], bound[b, :, h], lse_bound[b, h] = _attend(q[b, :, h], k, v, sees, scale, dtype)
    return out, lse, bound, lse_bound
