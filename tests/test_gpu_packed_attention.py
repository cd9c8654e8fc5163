"""packed_attention against the float64 oracle, on every element (MI355X): sequences from none
to long ones, with the mask and without, shared heads, head sizes, strides, rows outside all
sequences, infinities and NaN that a row does not see, streams and graphs."""
import numpy as np
import pytest
import torch

import bit_quantized_gemm_amd as w4
import oracle.request_ref as ref

from block_helpers import DEV, TORCH, assert_within, values_of

pytestmark = pytest.mark.gpu


def inputs(T, HQ, HKV, D, dtype, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed + T + HQ + D)
    joint = (torch.randn(T, HQ + 2 * HKV, D, generator=g) * std).to(TORCH[dtype]).to(DEV)
    return joint.split([HQ, HKV, HKV], 1)


def starts_of(lens, first=0):
    return torch.tensor([first + sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=DEV)


def padded(T, HQ, wide):
    """Tokens of a batch of T, or with so much padding behind them that 128-row tiles are taken."""
    return max(T, 23040 // HQ + 1) if wide else T


def check(q, k, v, starts, what, causal=True, scale=None):
    dtype = "f16" if q.dtype == torch.float16 else "bf16"
    out = torch.full_like(q, 3.0)
    got, lse = w4.packed_attention(q, k, v, starts, causal=causal, scale=scale, return_lse=True, out=out)
    y, ly, bound, lb, inside = ref.packed_attention_ref(*(values_of(t) for t in (q, k, v)), starts.cpu().numpy(), causal, scale, dtype)
    o, l = values_of(got), lse.double().cpu().numpy()
    assert_within(o[inside], y[inside], bound[inside], what)
    assert_within(l[:, inside], ly[:, inside], lb[:, inside], what + " lse")
    assert (o[~inside] == 3.0).all()
    return got


LENGTHS = [[1], [2, 1, 1], [31, 32, 33], [5, 0, 64, 0, 0, 127], [128, 129, 1], [257], [300, 7, 90, 1, 1, 200], [511, 513], [0, 0], [1000]]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens", LENGTHS, ids=lambda l: "-".join(map(str, l)))
def test_lengths(lens, causal, wide):
    T = sum(lens)
    for HQ, HKV, D, dtype in ((4, 2, 64, "bf16"), (3, 3, 128, "f16"), (8, 1, 40, "bf16")):
        print(f"case: {lens} {HQ}/{HKV} D{D} {dtype} causal {causal}", flush=True)
        q, k, v = inputs(padded(T + 9, HQ, wide), HQ, HKV, D, dtype)
        check(q, k, v, starts_of(lens, 4), f"{lens}", causal)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("D", range(8, 129, 8))
def test_head_sizes(D, wide):
    for dtype in ("bf16", "f16"):
        check(*inputs(padded(230, 6, wide), 6, 2, D, dtype), starts_of([150, 80]), f"D{D} {dtype}")


@pytest.mark.parametrize("HQ,HKV", [(1, 1), (7, 7), (5, 1), (24, 8), (16, 1), (33, 1), (64, 2), (130, 1)])
def test_shared_heads(HQ, HKV):
    """Groups that do and do not divide a tile's rows, and one with more heads than a tile."""
    for causal in (True, False):
        for wide in (True, False):
            check(*inputs(padded(333, HQ, wide), HQ, HKV, 72, "bf16"), starts_of([200, 3, 130]), f"{HQ}/{HKV}", causal)


def test_many_sequences():
    """More sequences than a wave has lanes, most of them short, some empty."""
    rng = np.random.default_rng(5)
    for count in (64, 65, 129, 400, 4096):
        lens = [int(n) for n in np.where(rng.random(count) < 0.2, 0, rng.integers(1, 12 if count < 4096 else 3, count))]
        lens[count // 2], lens[-1] = 300, 140
        check(*inputs(sum(lens) + 5, 4, 2, 64, "bf16"), starts_of(lens), f"{count} sequences")


def test_long():
    """One long sequence among short ones against the float64 form on the device, picked heads."""
    lens = [4352, 1, 2049, 333, 0, 77]
    T = sum(lens) + 50
    q, k, v = inputs(T, 24, 8, 128, "bf16")
    starts = starts_of(lens)
    for causal in (True, False):
        got = w4.packed_attention(q, k, v, starts, causal=causal)
        at = 0
        for n in lens:
            for h in (0, 13, 23):
                if not n:
                    continue
                a, b, c = (t[at:at + n, i].double() for t, i in ((q, h), (k, h // 3), (v, h // 3)))
                s = a @ b.t() * 128 ** -0.5
                if causal:
                    s.masked_fill_(torch.ones_like(s, dtype=torch.bool).triu(1), float("-inf"))
                p = torch.softmax(s, 1)
                # weights and out rounded: 2^-8 of sum p |v| each way, out's half spacing
                bound = 2 * (p @ c.abs()) * (2.0 ** -8 + 2.0 ** -14) + 2.0 ** -8 * (p @ c).abs() + 1e-30
                assert ((got[at:at + n, h].double() - p @ c).abs() <= bound).all(), (n, h)
            at += n


@pytest.mark.parametrize("starts", [[0, 50, 50, 200], [-5, 30, 1000], [20, 10, 100], [500, 600], [60, 60], [10, 90, 40, 120]])
def test_starts_that_leave_or_fall(starts):
    """Clamped; a sequence that ends before it starts is empty. (No two overlap but in the last, which only has to stay in bounds.)"""
    q, k, v = inputs(200, 4, 2, 64, "bf16")
    s = torch.tensor(starts, dtype=torch.int32, device=DEV)
    if starts == [10, 90, 40, 120]:
        out = torch.full_like(q, 3.0)
        w4.packed_attention(q, k, v, s, out=out)
        assert (out[:10] == 3.0).all() and (out[120:] == 3.0).all() and (out[10:40] != 3.0).any()
        return
    check(q, k, v, s, f"{starts}")


def test_strides():
    """Heads before tokens, slices of wider tensors, shared keys (head stride 0)."""
    T, HQ, HKV, D = 150, 6, 2, 40
    q, k, v = inputs(T, HQ, HKV, D, "bf16")
    starts = starts_of([100, 45])
    want = check(q, k, v, starts, "joint")
    qt = q.transpose(0, 1).contiguous().transpose(0, 1)
    wide = torch.full((T, HQ + 1, 2 * D), 9.0, device=DEV, dtype=torch.bfloat16)
    out = wide[:, :HQ, D:]
    got = w4.packed_attention(qt, k.clone(), v.clone(), starts, out=out)
    assert torch.equal(got[:145], want[:145]) and (got[145:] == 9.0).all()
    out[:145] = 9.0
    assert (wide == 9.0).all()
    one = w4.packed_attention(q, k[:, :1].expand(T, HKV, D), v[:, :1].expand(T, HKV, D), starts)
    assert torch.equal(one[:145], w4.packed_attention(q, k[:, :1], v[:, :1], starts)[:145])


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,HQ,HKV", [(64, 4, 2), (128, 3, 3), (72, 8, 1)])
def test_what_a_row_does_not_see(D, HQ, HKV, dtype, wide):
    """Infinities and NaN in later tokens, and in other sequences, change no earlier row; rows that see them say so."""
    lens = [70, 150, 260, 20]
    starts, T = starts_of(lens), sum(lens)
    q, k, v = inputs(padded(T, HQ, wide), HQ, HKV, D, dtype)
    y, _, bound, _, _ = ref.packed_attention_ref(*(values_of(t) for t in (q, k, v)), starts.cpu().numpy(), dtype=dtype)
    for tensor, token, value in ((v, 69, float("nan")), (v, 100, float("inf")), (k, 130, float("nan")), (v, 300, float("-inf")), (k, 400, float("inf")),
                                 (v, 480, float("nan")), (q, 222, float("nan"))):
        t = tensor.clone()
        t[token, :, D // 2] = value
        got = w4.packed_attention(*(t if s is tensor else s for s in (q, k, v)), starts)[:T]
        end = next(e for e in (70, 220, 480, 500) if token < e)
        others = torch.ones(T, dtype=torch.bool, device=DEV)
        others[token:(token + 1 if tensor is q else end)] = False
        rows = others.cpu().numpy()      # (those of the same tile take the slow way)
        assert_within(values_of(got)[rows], y[:T][rows], bound[:T][rows], f"{token} {value}")
        if tensor is v:
            assert not torch.isfinite(got[token:end, :, D // 2]).any()
            assert torch.isfinite(got[token:end, :, :D // 2]).all()
        elif tensor is q or value != value:
            assert got[~others].isnan().all()


@pytest.mark.parametrize("dtype,size", [("bf16", 1e4), ("bf16", 1e8), ("f16", 150.0), ("f16", 3e3)])
def test_large_scores(dtype, size):
    lens = [40, 200]
    for wide in (False, True):
        q, k, v = inputs(padded(240, 2, wide), 2, 2, 64, dtype, std=1.0)
        check((q.float() * size).to(q.dtype), k, v, starts_of(lens), f"{dtype} {size}", scale=1.0)


def test_past_32_bits():
    """Tokens so far apart that a sequence passes 2^32 bytes several times."""
    T, D, far = 1100, 64, 2**22
    space = torch.empty(2, T * far, dtype=torch.bfloat16, device=DEV)               # 9 GB each; the result in its own
    q, k, v = inputs(T, 4, 2, D, "bf16")
    starts = starts_of([5, 1000, 95])
    want = w4.packed_attention(q, k, v, starts)
    spread = [space[i // 3].as_strided((T, t.shape[1], D), (far, D, 1), i // 3 * T * far + 4096 * i) for i, t in enumerate((q, k, v, q))]
    for to, t in zip(spread, (q, k, v)):
        to.copy_(t)
    got = w4.packed_attention(*spread[:3], starts, out=spread[3])
    assert torch.equal(got, want)


def test_repeats_streams_and_graph():
    lens = [200, 0, 333, 1]
    q, k, v = inputs(540, 6, 2, 72, "bf16")
    starts = starts_of(lens)
    outs = [torch.zeros_like(q) for _ in range(4)]
    w4.packed_attention(q, k, v, starts, out=outs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    w4.packed_attention(q, k, v, starts, out=outs[1], stream=side)
    w4.packed_attention(q, k, v, starts, out=outs[2], stream=side.cuda_stream)
    w4.packed_attention(q, k, v, starts, out=outs[3])
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(o, outs[0]) for o in outs)
    hq, hs, ho = q.clone(), starts.clone(), torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w4.packed_attention(hq, k, v, hs, out=ho)
    for i in range(4):
        new = starts_of([50 * i, 540 - 50 * i - 7 * i, 3 * i])
        hs.copy_(torch.nn.functional.pad(new, (0, 1), value=int(new[-1])))
        hq.copy_(q * (i + 1))
        ho.zero_()
        g.replay()
        eager = w4.packed_attention(q * (i + 1), k, v, new, out=torch.zeros_like(q))
        torch.cuda.synchronize()
        assert torch.equal(ho, eager)
