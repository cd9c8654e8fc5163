"""Plain CPU oracles of the operators around the 4-bit layers, in float64:
MXFP4 quantisation, rotary positions over several axes, and attention to keys
of another length, each with the error bound its kernel is held to.

TEST INFRASTRUCTURE ONLY. The product (``bit_quantized_gemm_amd``) never
imports it and shares no code with it. (gemm_mxfp4_few's oracle is
gemm_mxfp4's, in w4a4_ref.py.)

16-bit tensors come as bit patterns (uint16) with dtype "bf16" or "f16".
"""
from __future__ import annotations

import numpy as np

from .quantize_ref import E2M1_MAGNITUDES, nearest_even_index
from .w4a4_ref import half_bits_to_f64

__all__ = ["quantize_mxfp4_ref", "lora_down_half", "rotary_ref", "rotary_bound", "attention_ref",
           "half_spacing"]


def quantize_mxfp4_ref(x_bits, dtype="bf16"):
    """x [M, K] -> (act uint8 [M, K/2], ascales uint8 [K/32, M]).

    Per block of 32: the largest magnitude amax gives the exponent
    floor(log2 amax) - 2, at least -127; the scale is that power of two; a code
    is the E2M1 magnitude nearest |x| / scale (ties to the even code,
    saturating at 6) and x's sign. Zero block: exponent -127. A NaN or an
    infinity: byte 255, codes 0."""
    x = half_bits_to_f64(np.asarray(x_bits, dtype=np.uint16), dtype)
    M, K = x.shape
    v = x.reshape(M, K // 32, 32)
    fine = np.isfinite(v).all(axis=-1)
    a = np.where(fine[..., None], np.abs(v), 0.0)
    amax = a.max(axis=-1)
    # frexp: amax = f * 2^e with f in [0.5, 1), so floor(log2 amax) = e - 1
    exp = np.where(amax > 0, np.frexp(amax)[1] - 1 - 2, -127)
    exp = np.maximum(exp, -127)
    codes = nearest_even_index(np.ldexp(a, -exp[..., None]), E2M1_MAGNITUDES)
    sign = np.signbit(v) & fine[..., None]
    codes = (codes + 8 * sign).astype(np.uint8).reshape(M, K)
    act = codes[:, 0::2] | (codes[:, 1::2] << 4)
    byte = np.where(fine, exp + 127, 255).astype(np.uint8)
    return act, np.ascontiguousarray(byte.T)


def lora_down_half(x_bits, down_bits, dtype):
    """(x @ down^T, sum |x down|) in float64."""
    x, d = half_bits_to_f64(x_bits, dtype), half_bits_to_f64(down_bits, dtype)
    return x @ d.T, np.abs(x) @ np.abs(d).T


def half_spacing(y, dtype):
    """Distance between neighbours of the 16-bit type at |y| (its smallest near zero)."""
    digits, least = (8, -133) if dtype == "bf16" else (11, -24)
    e = np.where(y == 0, -1000, np.frexp(np.abs(y))[1])
    return np.ldexp(1.0, np.maximum(e - digits, least))


def rotary_ref(x_bits, positions, inv_freq, sections, interleaved=True, inverse=False, dtype="bf16"):
    """x [B, L, H, D] bits, positions [B, L, axes] -> float64 [B, L, H, D]."""
    x = half_bits_to_f64(x_bits, dtype)
    out = x.copy()
    P = int(sum(sections))
    j = 0
    for axis, n in enumerate(sections):
        for _ in range(n):
            t = positions[..., axis].astype(np.float64) * np.float64(inv_freq[j])
            c, s = np.cos(t)[..., None], np.sin(t)[..., None]
            if inverse:
                s = -s
            i0, i1 = (2 * j, 2 * j + 1) if interleaved else (j, j + P)
            out[..., i0] = x[..., i0] * c - x[..., i1] * s
            out[..., i1] = x[..., i0] * s + x[..., i1] * c
            j += 1
    return out


def rotary_bound(x_bits, y, sections, interleaved, dtype):
    """Largest allowed |kernel - y|: half a spacing of the 16-bit type for the
    rounding, and 2^-17 (|u| + |w|) for the float32 arithmetic: the angle
    within 2^-22 turns (1.5e-6 rad), the sine and cosine within about as much
    again, four float32 roundings. Copied elements: 0."""
    x = np.abs(half_bits_to_f64(x_bits, dtype))
    P = int(sum(sections))
    mag = np.zeros_like(x)
    if interleaved:
        s = x[..., 0:2 * P:2] + x[..., 1:2 * P:2]
        mag[..., 0:2 * P:2] = s
        mag[..., 1:2 * P:2] = s
    else:
        s = x[..., :P] + x[..., P:2 * P]
        mag[..., :P] = s
        mag[..., P:2 * P] = s
    half = np.where(np.arange(x.shape[-1]) < 2 * P, 0.5 * half_spacing(y, dtype), 0.0)
    return half * (1 + 2.0 ** -6) + mag * 2.0 ** -17


def attention_ref(q_bits, k_bits, v_bits, kv_lens, scale, dtype="bf16"):
    """q [B, LQ, HQ, D], k and v [B, LK, HKV, D] bits -> (out [B, LQ, HQ, D],
    lse [B, HQ, LQ], bound on |kernel out - out|, bound on |kernel lse - lse|),
    float64. kv_lens: keys in use per sequence.

    The bounds: with T = sum p |v| / sum p, u the unit roundoff of the 16-bit
    type (2^-8 bf16, 2^-11 f16) and ds the largest float32 error of a score
    (D + 8 roundings of sum |q k| scale, and the exponent's own rounding of
    its argument, 2^-23 of the largest score's magnitude), a weight is off by
    at most u + 2 ds + 2^-20 relative, so out by that times 2 T (the sum it is
    divided by included), plus the output's half spacing; f16 weights below
    2^-14 are off by 2^-25 absolute, at most 2^-25 sum |v|."""
    q, k, v = (half_bits_to_f64(b, dtype) for b in (q_bits, k_bits, v_bits))
    B, LQ, HQ, D = q.shape
    HKV = k.shape[2]
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
    out, bound = np.zeros((B, LQ, HQ, D)), np.zeros((B, LQ, HQ, D))
    lse, lse_bound = np.full((B, HQ, LQ), -np.inf), np.zeros((B, HQ, LQ))
    for b in range(B):
        n = int(kv_lens[b])
        if n == 0:
            continue
        for h in range(HQ):
            g = h // (HQ // HKV)
            kk, vv = k[b, :n, g], v[b, :n, g]
            s = scale * (q[b, :, h] @ kk.T)
            top = s.max(axis=1, keepdims=True)
            p = np.exp(s - top)
            total = p.sum(axis=1, keepdims=True)
            o = p @ vv / total
            ds = (D + 8) * 2.0 ** -24 * (scale * (np.abs(q[b, :, h]) @ np.abs(kk).T)).max(axis=1, keepdims=True) \
                + 2.0 ** -22 * np.abs(s).max(axis=1, keepdims=True)
            T = p @ np.abs(vv) / total
            out[b, :, h] = o
            lse[b, h] = (top + np.log(total))[:, 0]
            tiny = 2.0 ** -25 * np.abs(vv).sum(axis=0) if dtype == "f16" else 0.0
            bound[b, :, h] = 2 * T * (u + 2 * ds + 2.0 ** -20) + 0.5 * half_spacing(o, dtype) * (1 + 2.0 ** -6) + tiny
            lse_bound[b, h] = (2 * ds)[:, 0] + 2.0 ** -20 * (1 + np.abs(lse[b, h]))
    return out, lse, bound, lse_bound
