"""Parity of cross_attention with the float64 oracle (MI355X) within the bounds
that oracle.block_ref.attention_ref derives."""
import numpy as np
import pytest
import torch

import bit_quantized_gemm_amd as w4
import oracle.block_ref as ref

from block_helpers import DEV, TORCH, assert_within, bits_of, half_bits, normal_bits, to_dev, values_of

pytestmark = pytest.mark.gpu


def inputs(rng, B, LQ, LK, HQ, HKV, D, dtype, std=1.0):
    return [normal_bits(rng, s, dtype, std) for s in ((B, LQ, HQ, D), (B, LK, HKV, D), (B, LK, HKV, D))]


def check(q, k, v, lens, dtype, what, scale=None, dev=None, **kw):
    D, LK = q.shape[-1], k.shape[1]
    dev = dev or [to_dev(t, dtype) for t in (q, k, v)]
    kl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
    out, lse = w4.cross_attention(*dev, kv_lens=kl, scale=scale, return_lse=True, **kw)
    use = [LK] * len(q) if lens is None else [min(max(n, 0), LK) for n in lens]
    y, ly, bound, lb = ref.attention_ref(q, k, v, use, D ** -0.5 if scale is None else scale, dtype)
    assert_within(values_of(out), y, bound, what)
    assert_within(lse.double().cpu().numpy(), ly, lb, what + " lse")
    return out, lse


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("B,LQ,LK,HQ,HKV,D", [
    (1, 1, 1, 1, 1, 8), (1, 1, 5, 1, 1, 64), (2, 1, 77, 4, 2, 128), (1, 3, 64, 2, 1, 40), (2, 31, 65, 3, 3, 72),
    (1, 32, 128, 2, 2, 96), (1, 33, 129, 2, 2, 64), (2, 100, 77, 4, 4, 128), (1, 128, 256, 2, 1, 104),
    (1, 129, 63, 3, 1, 80), (1, 255, 512, 2, 2, 128), (1, 257, 300, 1, 1, 88), (1, 300, 1, 2, 2, 16),
    (3, 17, 190, 8, 1, 24), (1, 1, 3000, 8, 8, 128), (2, 2, 1025, 24, 8, 128), (1, 513, 700, 2, 2, 48)])
def test_sizes(B, LQ, LK, HQ, HKV, D, dtype):
    print(f"case: {B} {LQ} {LK} {HQ} {HKV} {D} {dtype}", flush=True)
    rng = np.random.default_rng(B + LQ + LK + HQ + D)
    check(*inputs(rng, B, LQ, LK, HQ, HKV, D, dtype), None, dtype, f"{LQ}x{LK} D{D}")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("LQ,D,HQ,HKV", [(1, 128, 6, 2), (5, 64, 4, 4), (140, 72, 2, 2), (300, 128, 2, 1)])
def test_lengths(LQ, D, HQ, HKV, dtype):
    """Lengths of zero, one, around every tile edge, all, and out of range (taken as the
    nearest); memory past a length holds NaN and infinities and is never read."""
    lens = [0, 1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 500, 511, 512, -3, 600]
    rng = np.random.default_rng(LQ + D)
    q, k, v = inputs(rng, len(lens), LQ, 512, HQ, HKV, D, dtype)
    for b, n in enumerate(lens):
        for t in (k, v):
            t[b, max(n, 0):] = (0x7FC0 if b % 2 else 0x7F80) if dtype == "bf16" else (0x7E00 if b % 2 else 0xFC00)
    check(q, k, v, lens, dtype, f"lengths LQ={LQ}")


@pytest.mark.parametrize("B,HQ,HKV,LK", [(100, 2, 1, 700), (65, 3, 3, 520), (2, 8, 4, 6000), (7, 6, 2, 3000)])
@pytest.mark.parametrize("shape", ["falling", "one long", "random", "mostly empty"])
def test_uneven_sequences_of_one_token(B, HQ, HKV, LK, shape):
    """Sequences of very different lengths, whose keys are cut into parts of even length:
    every key is counted once, whatever the lengths."""
    rng = np.random.default_rng(B + LK)
    lens = {"falling": [LK * (B - b) // B for b in range(B)], "one long": [3] * (B - 1) + [LK],
            "random": [int(n) for n in rng.integers(0, LK + 1, B)],
            "mostly empty": [0 if b != B // 2 else LK for b in range(B)]}[shape]
    q, k, v = inputs(rng, B, 1, LK, HQ, HKV, 32, "f16")
    out, _ = check(q, k, v, lens, "f16", f"{B} {shape}")
    # counting: with equal keys the result is the mean of the values in use
    same = np.repeat(k[:1, :1], LK, 1).repeat(B, 0)
    count = half_bits(np.ones((B, LK, HKV, 32)) * (np.arange(LK) % 2)[None, :, None, None], "f16")
    check(q, same, count, lens, "f16", f"{B} {shape} counted")


@pytest.mark.parametrize("LQ", [1, 200])
def test_all_lengths_zero_and_no_keys(LQ):
    q = to_dev(normal_bits(np.random.default_rng(1), (2, LQ, 4, 64), "bf16"), "bf16")
    kv = torch.full((2, 96, 2, 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    for k, lens in ((kv, torch.zeros(2, dtype=torch.int32, device=DEV)), (kv[:, :0], None)):
        out, lse = w4.cross_attention(q, k, k, kv_lens=lens, return_lse=True)
        assert not out.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("LQ", [1, 8, 150])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_large_and_rising_scores(LQ, dtype):
    """Scores whose maximum rises along the keys (every tile rescales), and of a size
    where only the shift by the maximum keeps the exponentials finite."""
    rng = np.random.default_rng(2)
    q, k, v = inputs(rng, 1, LQ, 400, 2, 2, 64, dtype)
    kf = np.ones((1, 400, 2, 64)) * (np.arange(400) / 40.0)[None, :, None, None] + rng.standard_normal((1, 400, 2, 64)) * 0.1
    q = half_bits(np.abs(rng.standard_normal((1, LQ, 2, 64))) * 4, dtype)
    check(q, half_bits(kf, dtype), v, None, dtype, "rising")
    check(q, half_bits(kf[:, ::-1], dtype), v, None, dtype, "falling")
    check(q, half_bits(-kf * 8, dtype), v, [390], dtype, "very negative")


def test_special_values():
    """A NaN key poisons the rows that see it; a key at minus infinity has no weight; a row
    whose scores are all minus infinity gives 0."""
    rng = np.random.default_rng(3)
    for LQ in (2, 140):
        q, k, v = inputs(rng, 3, LQ, 100, 2, 2, 64, "bf16")
        q[..., 0] = 0x3F80                       # 1.0
        k[0, 40, 0, 5] = 0x7FC0
        k[1, 7, 1] = 0
        k[1, 7, 1, 0] = 0xFF80                   # the score of key 7 is -inf
        k[2, :, 0] = 0
        k[2, :, 0, 0] = 0xFF80
        q[2, :, 0, 1:] = 0x3F80
        out, lse = w4.cross_attention(*(to_dev(t, "bf16") for t in (q, k, v)), return_lse=True)
        o, l = out.float().cpu().numpy(), lse.cpu().numpy()
        assert np.isnan(o[0, :, 0]).all() and np.isnan(l[0, 0]).all() and not np.isnan(o[0, :, 1]).any()
        keep = [j for j in range(100) if j != 7]
        y, ly, bound, lb = ref.attention_ref(q[1:2, :, 1:], k[1:2, keep, 1:], v[1:2, keep, 1:], [99], 0.125)
        assert_within(values_of(out[1:2, :, 1:]), y, bound, "without the key at -inf")
        assert not o[2, :, 0].any() and np.isneginf(l[2, 0]).all()


@pytest.mark.parametrize("LQ", [2, 150])
def test_strides(LQ):
    """Heads before tokens, slices of joint projections, keys and values repeated over the
    batch with stride 0, out inside a larger tensor."""
    rng = np.random.default_rng(4)
    B, LK, H, D = 2, 150, 3, 40
    q, k, v = inputs(rng, B, LQ, LK, H, H, D, "bf16")
    qd = to_dev(q, "bf16").transpose(1, 2).contiguous().transpose(1, 2)
    kv = torch.full((B, LK, 2, H, D + 8), float("nan"), dtype=torch.bfloat16, device=DEV)
    kv[:, :, 0, :, :D], kv[:, :, 1, :, :D] = to_dev(k, "bf16"), to_dev(v, "bf16")
    big = torch.full((B, LQ, H + 1, D + 8), 3.0, dtype=torch.bfloat16, device=DEV)
    check(q, k, v, [150, 77], "bf16", "strided", dev=[qd, kv[:, :, 0, :, :D], kv[:, :, 1, :, :D]], out=big[:, :, :H, :D])
    assert (big[:, :, H] == 3).all() and (big[..., D:] == 3).all()
    one = [to_dev(t[:1], "bf16").expand(B, LK, H, D) for t in (k, v)]
    check(q, np.repeat(k[:1], B, 0), np.repeat(v[:1], B, 0), None, "bf16", "repeated", dev=[to_dev(q, "bf16")] + one)


@pytest.mark.parametrize("LQ", [1, 40, 300])
@pytest.mark.parametrize("LK,step", [(1, 0), (5, 0), (45, 0), (700, 0), (45, 8), (300, 8)])
def test_keys_that_share_memory(LQ, LK, step):
    """One key for all positions (stride 0) and rows that overlap (stride 8): positions past the
    length are not in the sums, with infinities among the values too, which 0 times would be NaN."""
    print(f"case: {LQ} {LK} {step}", flush=True)
    rng = np.random.default_rng(LQ + LK)
    D = 64
    q = normal_bits(rng, (2, LQ, 2, D), "f16")
    flat = [normal_bits(rng, (2, LK * step + D), "f16") for _ in range(2)]
    dev = [to_dev(t, "f16").as_strided((2, LK, 1, D), (t.shape[1], step, D, 1)) for t in flat]
    k, v = (np.stack([np.stack([t[b, i * step:i * step + D] for i in range(LK)]) for b in range(2)])[:, :, None] for t in flat)
    lens = [LK, LK - LK // 3]
    check(q, k, v, lens, "f16", f"stride {step}", dev=[to_dev(q, "f16"), *dev])
    for t, host in zip(flat[1], v):      # the first position's first value: infinite
        t[0] = host[0, 0, 0] = 0x7C00
        for i in range(1, LK if step == 0 else 1):
            host[i, 0, 0] = 0x7C00
    vd = to_dev(flat[1], "f16").as_strided((2, LK, 1, D), (flat[1].shape[1], step, D, 1))
    out = w4.cross_attention(to_dev(q, "f16"), dev[0], vd, kv_lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    assert torch.isposinf(out[..., 0]).all() and torch.isfinite(out[..., 1:]).all()


def test_parts_join():
    """Attention over two parts of the keys joined by their log-sum-exps is attention over all."""
    rng = np.random.default_rng(5)
    q, k, v = inputs(rng, 1, 40, 300, 2, 2, 64, "f16")
    d = [to_dev(t, "f16") for t in (q, k, v)]
    (o1, l1), (o2, l2) = (w4.cross_attention(d[0], d[1][:, s], d[2][:, s], return_lse=True) for s in (slice(0, 111), slice(111, 300)))
    w = torch.softmax(torch.stack([l1, l2]), 0).permute(0, 1, 3, 2)[..., None]
    y, _, bound, _ = ref.attention_ref(q, k, v, [300], 0.125, "f16")
    got = (o1.float() * w[0] + o2.float() * w[1]).double().cpu().numpy()
    assert_within(got, y, 2 * bound, "joined")


def test_long_cache_past_32_bits():
    """A token stride that puts the last keys more than 2^32 bytes from the first."""
    B, LK, D = 1, 700, 128
    rng = np.random.default_rng(6)
    q, k, v = inputs(rng, B, 4, LK, 1, 1, D, "bf16")
    stride = (1 << 22) + 8
    buf = torch.empty(LK * stride, dtype=torch.bfloat16, device=DEV)
    kd = buf.as_strided((B, LK, 1, D), (LK * stride, stride, D, 1))
    vd = buf.as_strided((B, LK, 1, D), (LK * stride, stride, D, 1), 1 << 20)
    kd.copy_(to_dev(k, "bf16"))
    vd.copy_(to_dev(v, "bf16"))
    check(q, k, v, None, "bf16", "long", dev=[to_dev(q, "bf16"), kd, vd])
    q2 = normal_bits(rng, (B, 130, 1, D), "bf16")
    check(q2, k, v, [650], "bf16", "long, many rows", dev=[to_dev(q2, "bf16"), kd, vd])


def test_repeatable_other_stream_and_graph():
    rng = np.random.default_rng(7)
    for LQ in (1, 260):
        q, k, v = (to_dev(t, "bf16") for t in inputs(rng, 2, LQ, 1500, 4, 2, 128, "bf16"))
        lens = torch.tensor([1500, 900], dtype=torch.int32, device=DEV)
        want = w4.cross_attention(q, k, v, lens)
        for _ in range(3):
            assert torch.equal(want, w4.cross_attention(q, k, v, lens))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = w4.cross_attention(q, k, v, lens, stream=side)
        side.synchronize()
        assert torch.equal(want, got)
        sq, sl = q.clone(), lens.clone()
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            kept = w4.cross_attention(sq, k, v, sl)
        for i in range(4):
            sq.copy_(q * (i + 1))
            sl.copy_(lens - 100 * i)
            g.replay()
            eager = w4.cross_attention(q * (i + 1), k, v, lens - 100 * i)
            torch.cuda.synchronize()
            assert torch.equal(kept, eager)


def test_empty():
    for shape in ((0, 3, 2, 64), (2, 0, 2, 64), (2, 3, 0, 64)):
        q = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
        k = torch.empty((shape[0], 5, 2, 64), dtype=torch.bfloat16, device=DEV)
        assert w4.cross_attention(q, k, k).shape == shape
