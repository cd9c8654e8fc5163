"""Workspaces of the block operators through the C entry points (MI355X): of exactly the
stated size, in the middle of a larger buffer, holding zeros or all ones (NaN as float32).
Results are the same bytes whatever they held, within the oracle's bounds, and nothing around
workspace or outputs changes."""
import numpy as np
import pytest
import torch

import bit_quantized_gemm_amd as w4
import oracle.block_ref as ref
import oracle.w4a4_ref as gref

from block_helpers import DEV, assert_within, bits_of, normal_bits, to_dev, values_of

pytestmark = pytest.mark.gpu
EDGE = 4096
FILLS = (0x00, 0xFF, 0x5A)


class Guarded:
    """`n` bytes on the device with EDGE bytes of a pattern on both sides."""

    def __init__(self, n):
        self.n, self.all = n, torch.full((n + 2 * EDGE,), 0xA5, dtype=torch.uint8, device=DEV)
        self.bytes = self.all[EDGE:EDGE + n]
        self.ptr = self.bytes.data_ptr()

    def check(self, what):
        assert (self.all[:EDGE] == 0xA5).all() and (self.all[EDGE + self.n:] == 0xA5).all(), what + ": written outside"


def quantize(x, down, M, K, R, f16, fill):
    need = w4.quantize_mxfp4_workspace(M, K, R)
    ws, outs = Guarded(need), [Guarded(n) for n in (M * K // 2, K // 32 * M, M * R * 2)]
    ws.bytes.fill_(fill)
    for o in outs:
        o.bytes.fill_(fill)
    rc = w4.quantize_mxfp4_raw(f16, x.data_ptr(), down.data_ptr(), *(o.ptr for o in outs), M, K, R, ws.ptr, need,
                               torch.cuda.current_stream().cuda_stream)
    assert rc == w4.OK
    torch.cuda.synchronize()
    for g, what in zip([ws] + outs, ("workspace", "act", "ascales", "lora_act_in")):
        g.check(what)
    return need, [o.bytes.cpu().numpy() for o in outs]


@pytest.mark.parametrize("M,K,R,dtype", [(1, 12288, 1, "bf16"), (16, 12288, 33, "f16"), (37, 12288, 24, "bf16"), (129, 8224, 128, "f16"),
                                         (300, 4128, 17, "bf16"), (1001, 12288, 128, "bf16"), (700, 4128, 31, "f16"), (2049, 8224, 31, "bf16")])
def test_producer_in_slices(M, K, R, dtype):
    print(f"case: {M}x{K} R={R} {dtype}", flush=True)
    rng = np.random.default_rng(M + K + R)
    xb, db = normal_bits(rng, (M, K), dtype), normal_bits(rng, (R, K), dtype, 0.02)
    x, down = to_dev(xb, dtype), to_dev(db, dtype)
    first = None
    for fill in FILLS:
        need, got = quantize(x, down, M, K, R, dtype == "f16", fill)
        assert need > 0 and (first is None or all(np.array_equal(a, b) for a, b in zip(first, got)))
        first = got
    act, asc = ref.quantize_mxfp4_ref(xb, dtype)
    assert np.array_equal(first[0].reshape(act.shape), act) and np.array_equal(first[1].reshape(asc.shape), asc)
    y, T = ref.lora_down_half(xb, db, dtype)
    assert gref.check_output(first[2].view(np.uint16).reshape(M, R), y, T, dtype)["ok"]


def attend(q, k, v, lens, dtype, fill):
    """(workspace bytes, out, lse) of a call on dense tensors."""
    B, LQ, HQ, D = q.shape
    a = w4.AttentionArgs()
    for f, t in (("q_stride", q), ("k_stride", k), ("v_stride", v), ("out_stride", q)):
        for i in range(3):
            getattr(a, f)[i] = t.stride(i)
    a.batch, a.q_len, a.kv_len, a.q_heads, a.kv_heads, a.head_dim = B, LQ, k.shape[1], HQ, k.shape[2], D
    a.scale, a.f16 = D ** -0.5, int(dtype == "f16")
    kl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
    a.kv_lens = None if lens is None else kl.data_ptr()
    need = w4.cross_attention_workspace(a)
    ws, out, lse = Guarded(need), Guarded(q.numel() * 2), Guarded(B * HQ * LQ * 4)
    for g in (ws, out, lse):
        g.bytes.fill_(fill)
    a.q, a.k, a.v, a.out, a.lse = q.data_ptr(), k.data_ptr(), v.data_ptr(), out.ptr, lse.ptr
    a.workspace, a.workspace_bytes = ws.ptr, need
    assert w4.cross_attention_raw(a, torch.cuda.current_stream().cuda_stream) == w4.OK
    torch.cuda.synchronize()
    for g, what in ((ws, "workspace"), (out, "out"), (lse, "lse")):
        g.check(what)
    return need, out.bytes.view(q.dtype).view(q.shape), lse.bytes.view(torch.float32).view(B, HQ, LQ)


def lengths(shape, B, LK):
    return {"all": None, "falling": [LK * (B - b) // B for b in range(B)], "one long": [3] * (B - 1) + [LK],
            "mostly empty": [0 if b != B // 2 else LK for b in range(B)], "empty": [0] * B, "past the ends": [-7] * (B - 1) + [LK + 9],
            "random": [int(n) for n in np.random.default_rng(B + LK).integers(0, LK + 1, B)]}[shape]


@pytest.mark.parametrize("shape", ["all", "falling", "one long", "mostly empty", "empty", "past the ends", "random"])
@pytest.mark.parametrize("B,LQ,LK,HQ,HKV,D,dtype", [
    (7, 1, 3000, 6, 2, 32, "f16"), (2, 1, 6000, 8, 4, 128, "bf16"), (100, 1, 700, 2, 1, 40, "f16"), (65, 2, 520, 3, 3, 72, "bf16"),
    (3, 140, 1500, 2, 2, 64, "f16"), (2, 200, 1100, 4, 2, 128, "bf16"), (3, 130, 520, 2, 1, 72, "f16")])
def test_attention_in_parts(B, LQ, LK, HQ, HKV, D, dtype, shape):
    """Few rows (of several sequences: parts of even length) and 128-row tiles, keys cut."""
    lens = lengths(shape, B, LK)
    print(f"case: {B} {LQ}x{LK} {HQ}/{HKV} D{D} {dtype} {shape}", flush=True)
    rng = np.random.default_rng(B + LQ + LK)
    bits = [normal_bits(rng, s, dtype) for s in ((B, LQ, HQ, D), (B, LK, HKV, D), (B, LK, HKV, D))]
    dev = [to_dev(t, dtype) for t in bits]
    first = None
    for fill in FILLS:
        need, out, lse = attend(*dev, lens, dtype, fill)
        got = bits_of(out), lse.cpu().numpy()
        assert need > 0 and (first is None or (np.array_equal(first[0], got[0]) and np.array_equal(first[1], got[1])))
        first = got
    use = [LK] * B if lens is None else [min(max(n, 0), LK) for n in lens]
    y, ly, bound, lb = ref.attention_ref(*bits, use, D ** -0.5, dtype)
    assert_within(values_of(out), y, bound, shape)
    assert_within(first[1].astype(np.float64), ly, lb, shape + " lse")


@pytest.mark.parametrize("lens", ["all", "falling", "mostly empty"])
@pytest.mark.parametrize("B,LQ,LK,HQ,HKV,D,dtype", [
    (3, 1200, 600, 9, 9, 64, "bf16"),      # 128-row tiles: 256 whole, 14 cut in two
    (1, 2100, 1030, 17, 17, 72, "f16"),    # 289: 256 whole, 33 cut in four
    (2, 700, 520, 24, 24, 128, "bf16"),    # 288: 256 whole, 32 cut in two
    (100, 1, 1300, 6, 3, 128, "f16"),      # the few-row kernel: 256 whole, 44 cut in five
    (10, 5, 600, 30, 30, 40, "bf16")])     # likewise, 44 in two
def test_whole_and_cut_tiles_in_one_launch(B, LQ, LK, HQ, HKV, D, dtype, lens):
    """More tiles than compute units: the first 256 are done whole, the keys of the rest are cut, and joined by a second launch."""
    print(f"case: {B} {LQ}x{LK} {HQ}/{HKV} D{D} {dtype} {lens}", flush=True)
    lens = lengths(lens, B, LK)
    rng = np.random.default_rng(B + LQ + LK)
    bits = [normal_bits(rng, s, dtype) for s in ((B, LQ, HQ, D), (B, LK, HKV, D), (B, LK, HKV, D))]
    need, out, lse = attend(*(to_dev(t, dtype) for t in bits), lens, dtype, 0xFF)
    rows = LQ * (HQ // HKV)
    tile = 32 if rows <= 32 else 128
    tiles = -(-rows // tile) * B * HKV
    parts = min(256 // (tiles % 256), LK // 256)
    assert tiles > 256 and parts > 1 and need == (tiles % 256) * parts * tile * (D + 2) * 4      # the plan this is about
    y, ly, bound, lb = ref.attention_ref(*bits, [LK] * B if lens is None else lens, D ** -0.5, dtype)
    assert_within(values_of(out), y, bound, "out")
    assert_within(lse.double().cpu().numpy(), ly, lb, "lse")
