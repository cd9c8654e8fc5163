"""paged_attention against the float64 oracle, on every element (MI355X): page sizes, tables,
lengths, several new tokens, entries that are no page, what a row does not see, caches past 32 bits,
workspaces, streams and graphs; and with cache_append, token by token, against packed_attention."""
import numpy as np
import pytest
import torch

import bit_quantized_gemm_amd as w4
import oracle.request_ref as ref

from block_helpers import DEV, TORCH, assert_within, values_of

pytestmark = pytest.mark.gpu


def inputs(B, Q, HQ, HKV, D, page, lens, dtype, seed=0, spare=2):
    """q, caches whose unused places are NaN, table, lens."""
    g = torch.Generator().manual_seed(seed + B + 3 * page + D)
    use = [-(-max(n, 0) // page) for n in lens]
    pages = sum(use) + spare
    q = torch.randn(B, Q, HQ, D, generator=g).to(TORCH[dtype]).to(DEV)
    kc, vc = (torch.full((pages, page, HKV, D), float("nan")) for _ in range(2))
    order, table, at = torch.randperm(pages, generator=g).to(torch.int32), torch.full((B, max(use + [1]) + 1), -1, dtype=torch.int32), 0
    for b, n in enumerate(lens):
        for i in range(use[b]):
            e = int(order[at])
            table[b, i] = e
            m = min(page, n - i * page)
            for c in (kc, vc):
                c[e, :m] = torch.randn(m, HKV, D, generator=g)
            at += 1
    return q, kc.to(TORCH[dtype]).to(DEV), vc.to(TORCH[dtype]).to(DEV), table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)


def check(q, kc, vc, table, lens, what, **kw):
    dtype = "f16" if q.dtype == torch.float16 else "bf16"
    got, lse = w4.paged_attention(q, kc, vc, table, lens, return_lse=True, **kw)
    y, ly, bound, lb = ref.paged_attention_ref(*(values_of(t) for t in (q, kc, vc)), table.cpu().numpy(), lens.cpu().numpy(), dtype=dtype,
                                               **{k: v for k, v in kw.items() if k == "scale"})
    assert_within(values_of(got), y, bound, what)
    assert_within(lse.double().cpu().numpy(), ly, lb, what + " lse")
    return got, lse


@pytest.mark.parametrize("page", [16, 32, 48, 64, 80, 128, 272, 1008])
def test_page_sizes(page):
    for lens in ([1, 15, 16, 17, 0], [page, page + 1, page - 1, 2 * page], [1000, 3, 700]):
        for HQ, HKV, D, dtype in ((6, 2, 64, "bf16"), (3, 3, 128, "f16")):
            print(f"case: page {page} {lens} {HQ}/{HKV} D{D} {dtype}", flush=True)
            check(*inputs(len(lens), 1, HQ, HKV, D, page, lens, dtype), f"page {page} {lens}")


@pytest.mark.parametrize("D", range(8, 129, 8))
def test_head_sizes(D):
    for dtype in ("bf16", "f16"):
        check(*inputs(2, 1, 8, 2, D, 16, [333, 50], dtype), f"D{D} {dtype}")


@pytest.mark.parametrize("Q", [2, 3, 8, 17, 33, 70])
@pytest.mark.parametrize("HQ,HKV", [(4, 4), (12, 4), (16, 1)])
def test_several_new_tokens(Q, HQ, HKV):
    """Each sees the keys up to its own; sequences shorter than the new tokens leave the first without any."""
    for lens in ([Q, Q + 40, 500, Q - 1, 0, 1], [700, 300]):
        check(*inputs(len(lens), Q, HQ, HKV, 72, 32, lens, "bf16"), f"{Q} tokens {lens}")


@pytest.mark.parametrize("B,lens", [(1, "full"), (1, "short"), (3, "falling"), (40, "any"), (100, "any"), (300, "any")])
def test_batches_and_parts(B, lens):
    """Tiles that are cut, whole, and both; a table far wider than the lengths."""
    rng = np.random.default_rng(B)
    n = {"full": [3000], "short": [40], "falling": [2500, 1200, 10], "any": [int(x) for x in rng.integers(0, 700 if B < 100 else 90, B)]}[lens]
    q, kc, vc, table, l = inputs(B, 1, 8, 4, 64, 16, n, "bf16")
    wide = torch.full((B, 400), 2**30, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    a = check(q, kc, vc, wide, l, f"{B} {lens}")
    b = check(q, kc, vc, table, l, f"{B} {lens}")
    assert torch.isfinite(a[0]).all() and torch.isfinite(b[0]).all()


@pytest.mark.parametrize("Q", [1, 4])
def test_entries_that_are_no_page(Q):
    for bad in (-1, 2**31 - 1, -2**31, 10**6):
        q, kc, vc, table, lens = inputs(3, Q, 6, 2, 64, 16, [400, 90, 33], "bf16")
        table[0, 3], table[0, 24], table[1, 0] = bad, bad, bad
        table[2, :] = bad                                      # a sequence without a page: no keys
        got, lse = check(q, kc, vc, table, lens, f"{bad}")
        assert (got[2] == 0).all() and (lse[2] == float("-inf")).all()
    check(q, kc, vc, table, torch.tensor([2**31 - 1, -5, 2**30], dtype=torch.int32, device=DEV), "lengths past the table")


def test_what_a_row_does_not_see():
    """Infinities and NaN in the newest tokens' own keys and values change no earlier one of them."""
    for dtype in ("bf16", "f16"):
        q, kc, vc, table, lens = inputs(2, 4, 6, 2, 72, 16, [200, 35], dtype)
        want = w4.paged_attention(q, kc, vc, table, lens)
        y, _, bound, _ = ref.paged_attention_ref(*(values_of(t) for t in (q, kc, vc)), table.cpu().numpy(), [200, 35], dtype=dtype)
        for value in (float("nan"), float("inf")):
            for cache, i in ((vc, 3), (vc, 1), (kc, 2)):
                c = cache.clone()
                key = 200 - 4 + i
                c[table[0, key // 16].long(), key % 16, :, 5] = value
                got = w4.paged_attention(q, c if cache is kc else kc, c if cache is vc else vc, table, lens)
                assert_within(values_of(got)[0, :i], y[0, :i], bound[0, :i], f"{value} in new token {i}")
                assert torch.equal(got[1], want[1])
                if cache is vc:
                    assert not torch.isfinite(got[0, i:, :, 5]).any() and torch.isfinite(got[0, i:, :, 6:]).all()


def test_strides():
    """Keys and values as slices of one cache, heads before places, strided q and out, a table of a wider one."""
    q, kc, vc, table, lens = inputs(3, 2, 6, 2, 40, 16, [100, 30, 77], "bf16")
    want = w4.paged_attention(q, kc, vc, table, lens)
    joint = torch.stack([kc, vc], 1).transpose(2, 3).contiguous().transpose(2, 3)
    wq = torch.zeros(3, 2, 9, 48, dtype=torch.bfloat16, device=DEV)
    wq[:, :, 1:7, 8:] = q
    wt = torch.full((3, table.shape[1] + 5), 7, dtype=torch.int32, device=DEV)
    wt[:, 2:2 + table.shape[1]] = table
    out = torch.full((2, 3, 7, 40), 5.0, dtype=torch.bfloat16, device=DEV)
    view = out.transpose(0, 1)[:, :, :6]
    got = w4.paged_attention(wq[:, :, 1:7, 8:], joint[:, 0], joint[:, 1], wt[:, 2:2 + table.shape[1]], lens, out=view)
    assert torch.equal(got, want) and got.data_ptr() == out.data_ptr() and (out[:, :, 6] == 5.0).all()


def test_past_32_bits():
    """A cache of more than 2^32 bytes, and pages on both sides of every such border."""
    H, D, page = 8, 128, 64
    pages = 2**33 // (2 * H * D * page) + 3
    kc, vc = (torch.full((pages, page, H, D), float("nan"), dtype=torch.float16, device=DEV) for _ in range(2))
    border = 2**32 // (2 * H * D * page)
    table = torch.tensor([[0, border - 1, border, 2 * border, pages - 1]], dtype=torch.int32, device=DEV)
    n = 5 * page - 3
    k, v = (torch.randn(n, H, D, device=DEV).half() for _ in range(2))
    at = torch.arange(n, device=DEV)
    w4.cache_append(k, v, kc, vc, table[0, at // page].long() * page + at % page)
    q = torch.randn(1, 2, H, D, device=DEV).half()
    got = w4.paged_attention(q, kc, vc, table, torch.tensor([n], dtype=torch.int32, device=DEV))
    small = torch.full((5, page, H, D), float("nan"), dtype=torch.float16, device=DEV)
    kc2, vc2 = small.clone(), small.clone()
    w4.cache_append(k, v, kc2, vc2, at)
    check(q, kc2, vc2, torch.arange(5, dtype=torch.int32, device=DEV)[None], torch.tensor([n], dtype=torch.int32, device=DEV), "small")
    want = w4.paged_attention(q, kc2, vc2, torch.arange(5, dtype=torch.int32, device=DEV)[None], torch.tensor([n], dtype=torch.int32, device=DEV))
    assert torch.equal(got, want)


def test_workspace_between_guards():
    for B, Q, n in ((1, 1, 5000), (8, 1, 3000), (3, 3, 900), (70, 1, 600)):
        q, kc, vc, table, lens = inputs(B, Q, 8, 4, 64, 16, [max(0, n - 37 * b) for b in range(B)], "bf16")
        want = w4.paged_attention(q, kc, vc, table, lens, return_lse=True)
        for fill in (0x00, 0xFF, 0x5A):
            out, lse = torch.empty_like(q), torch.empty_like(want[1])
            a = w4.PagedAttentionArgs()
            a.q, a.k_cache, a.v_cache, a.out, a.lse, a.table, a.lens = (t.data_ptr() for t in (q, kc, vc, out, lse, table, lens))
            a.batch, a.q_len, a.q_heads, a.kv_heads, a.head_dim = B, Q, 8, 4, 64
            a.pages, a.page_size, a.table_width, a.table_stride, a.scale = kc.shape[0], 16, table.shape[1], table.shape[1], 0.125
            for f, t in (("q_stride", q), ("k_stride", kc), ("v_stride", vc), ("out_stride", out)):
                for i in range(3):
                    getattr(a, f)[i] = t.stride(i)
            need = w4.paged_attention_workspace(a)
            buf = torch.full((need + 8192,), 0xA5, dtype=torch.uint8, device=DEV)
            buf[4096:4096 + need] = fill
            a.workspace, a.workspace_bytes = buf.data_ptr() + 4096, need
            assert need > 0 and w4.paged_attention_raw(a, torch.cuda.current_stream().cuda_stream) == w4.OK
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
            assert (buf[:4096] == 0xA5).all() and (buf[4096 + need:] == 0xA5).all()


def test_prompts_then_tokens():
    """Prompts packed and appended to the cache, then token by token: each step gives what one packed call over all tokens gives."""
    H, G, D, page, steps = 2, 3, 64, 16, 20
    lens = [50, 1, 129]
    B = len(lens)
    g = torch.Generator(device=DEV).manual_seed(1)
    full = [tuple(torch.randn(n + steps, h, D, generator=g, device=DEV).bfloat16() for h in (H * G, H, H)) for n in lens]
    table = torch.randperm(40, generator=g, device=DEV).to(torch.int32)[:36].view(B, 12)
    kc, vc = (torch.full((40, page, H, D), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))

    def slots(b, at):
        return table[b, at // page].long() * page + at % page
    q, k, v = (torch.cat([f[i][:n] for f, n in zip(full, lens)]) for i in range(3))
    w4.cache_append(k, v, kc, vc, torch.cat([slots(b, torch.arange(n, device=DEV)) for b, n in enumerate(lens)]))
    starts = torch.tensor([0, 50, 51, 180], dtype=torch.int32, device=DEV)
    first = w4.packed_attention(q, k, v, starts)
    all_starts = torch.tensor([0, 70, 91, 240], dtype=torch.int32, device=DEV)
    want = w4.packed_attention(*(torch.cat([f[i] for f in full]) for i in range(3)), all_starts).float()
    at = 0
    for b, n in enumerate(lens):
        lo = int(all_starts[b])
        assert (first[at:at + n].float() - want[lo:lo + n]).abs().max() < 0.02
        at += n
    for s in range(steps):
        now = torch.tensor([n + s for n in lens], device=DEV)
        q, k, v = (torch.stack([f[i][n + s] for f, n in zip(full, lens)]) for i in range(3))
        w4.cache_append(k, v, kc, vc, torch.cat([slots(b, now[b:b + 1]) for b in range(B)]))
        out = w4.paged_attention(q[:, None], kc, vc, table, (now + 1).to(torch.int32))[:, 0].float()
        for b, n in enumerate(lens):
            # two roundings of out and of the weights, twice: 4 * 2^-8 of values below 4
            assert (out[b] - want[int(all_starts[b]) + n + s]).abs().max() < 0.0625


def test_repeats_streams_and_graph():
    q, kc, vc, table, lens = inputs(8, 1, 8, 2, 128, 32, [2000, 900, 33, 0, 1500, 64, 5, 700], "bf16")
    want = w4.paged_attention(q, kc, vc, table, lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [w4.paged_attention(q, kc, vc, table, lens, stream=s) for s in (side, None, side.cuda_stream, None)]
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in got)
    hq, hl, ht = q.clone(), lens.clone(), table.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = w4.paged_attention(hq, kc, vc, ht, hl)
        again = w4.paged_attention(hq * 2, kc, vc, ht, hl)      # a second call's workspace in the same graph
    for i in range(4):
        swap = torch.randperm(8, generator=torch.Generator().manual_seed(i)).to(DEV)
        hl.copy_(lens[swap])
        ht.copy_(table[swap])
        hq.copy_(q * (1 + i))
        g.replay()
        eager = [w4.paged_attention(hq * f, kc, vc, ht, hl) for f in (1, 2)]
        torch.cuda.synchronize()
        assert torch.equal(kept, eager[0]) and torch.equal(again, eager[1])


@pytest.mark.parametrize("page", [16, 48, 128])
@pytest.mark.parametrize("Q,HQ,HKV,D,dtype", [(40, 4, 4, 128, "bf16"), (129, 3, 3, 64, "f16"), (300, 6, 2, 96, "bf16"), (65, 16, 1, 40, "f16"),
                                              (257, 2, 1, 128, "f16"), (33, 5, 5, 8, "bf16")])
def test_long_pieces_of_prompts(Q, HQ, HKV, D, dtype, page):
    """Many new tokens over a cache that holds more, just them, fewer or none."""
    for lens in ([Q + 700, Q, Q - 20, 0], [Q + 1], [Q + 31, Q + 1500]):
        print(f"case: {Q} {HQ}/{HKV} D{D} page {page} {lens} {dtype}", flush=True)
        check(*inputs(len(lens), Q, HQ, HKV, D, page, lens, dtype), f"{Q} {lens}")


def test_long_pieces_over_a_wide_table():
    """A table past the length from which on parts are even, and more tiles than compute units."""
    for B, lens in ((1, [6000]), (2, [5000, 100]), (40, [150 + 7 * b for b in range(40)])):
        q, kc, vc, table, l = inputs(B, 140, 8, 4, 64, 16, lens, "bf16")
        wide = torch.full((B, 600), 2**30, dtype=torch.int32, device=DEV)
        wide[:, :table.shape[1]] = table
        check(q, kc, vc, wide, l, f"{lens[:2]}")
        check(q, kc, vc, table, l, f"{lens[:2]}")


def test_long_pieces_with_entries_that_are_no_page():
    for bad in (-1, 2**31 - 1, -2**31, 10**6):
        for D in (64, 128):
            q, kc, vc, table, lens = inputs(3, 50, 6, 2, D, 16, [1400, 90, 70], "bf16")
            table[0, 3], table[0, 70], table[0, 87], table[1, 0] = bad, bad, bad, bad
            table[2, :] = bad
            got, lse = check(q, kc, vc, table, lens, f"{bad}")
            assert (got[2] == 0).all() and (lse[2] == float("-inf")).all()
        check(q, kc, vc, table, torch.tensor([2**31 - 1, -5, 2**30], dtype=torch.int32, device=DEV), "lengths past the table")


@pytest.mark.parametrize("Q,HQ,HKV", [(20, 6, 2), (150, 6, 2)])
def test_what_a_row_of_many_does_not_see(Q, HQ, HKV):
    """Infinities and NaN in a new token's key or value change no earlier one, with every entry a page and with one that is none."""
    for dtype in ("bf16", "f16"):
        for hole in (False, True):
            q, kc, vc, table, lens = inputs(2, Q, HQ, HKV, 72, 16, [Q + 200, Q + 5], dtype)
            if hole:
                table[:, 2] = -1
            y, _, bound, _ = ref.paged_attention_ref(*(values_of(t) for t in (q, kc, vc)), table.cpu().numpy(), lens.cpu().numpy(), dtype=dtype)
            want = w4.paged_attention(q, kc, vc, table, lens)
            for value in (float("nan"), float("inf")):
                for cache, i in ((vc, Q - 1), (vc, 7), (kc, 11)):
                    c, key = cache.clone(), 200 + i
                    c[table[0, key // 16].long(), key % 16, :, 5] = value
                    got = w4.paged_attention(q, c if cache is kc else kc, c if cache is vc else vc, table, lens)
                    assert_within(values_of(got)[0, :i], y[0, :i], bound[0, :i], f"{value} in new token {i}")
                    assert torch.equal(got[1], want[1])
                    if cache is vc:
                        assert not torch.isfinite(got[0, i:, :, 5]).any() and torch.isfinite(got[0, i:, :, 6:]).all()


def test_a_piece_is_the_packed_prompt():
    """A prompt as new tokens of an empty cache, whole and in pieces, within the roundings of the packed one; replayed."""
    T, HQ, HKV, D, page = 900, 8, 2, 128, 64
    q, kc, vc, table, lens = inputs(1, T, HQ, HKV, D, page, [T], "bf16")
    whole, _ = check(q, kc, vc, table, lens, "whole")
    y, _, bound, _ = ref.paged_attention_ref(*(values_of(t) for t in (q, kc, vc)), table.cpu().numpy(), lens.cpu().numpy(), dtype="bf16")
    for at, to in ((0, 300), (300, 337), (337, 900)):
        piece = w4.paged_attention(q[:, at:to], kc, vc, table, torch.tensor([to], dtype=torch.int32, device=DEV))
        assert_within(values_of(piece), y[:, at:to], bound[:, at:to], f"{at} to {to}")
    flat = torch.cat([c[table[0, :15].long()].reshape(-1, HKV, D)[:T][None] for c in (kc, vc)])
    packed = w4.packed_attention(q[0], flat[0].contiguous(), flat[1].contiguous(), torch.tensor([0, T], dtype=torch.int32, device=DEV))
    assert_within(values_of(packed), y[0], bound[0], "packed")
    hq, hl = q.clone(), lens.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = w4.paged_attention(hq, kc, vc, table, hl)
    for i in range(3):
        hq.copy_(q * (1 + i))
        hl.fill_(T - 200 * i)
        g.replay()
        eager = w4.paged_attention(hq, kc, vc, table, hl)
        torch.cuda.synchronize()
        assert torch.equal(kept, eager)


def test_long_pieces_past_32_bits_and_strided():
    """Pages on both sides of every 2^32-byte border of a cache, keys and values side by side, heads before places."""
    H, D, page, Q = 4, 72, 32, 90
    n = 5 * page - 3
    k, v = (torch.randn(n, H, D, device=DEV).half() for _ in range(2))
    at, lens = torch.arange(n, device=DEV), torch.tensor([n], dtype=torch.int32, device=DEV)
    kc, vc = (torch.full((5, page, H, D), float("nan"), dtype=torch.float16, device=DEV) for _ in range(2))
    w4.cache_append(k, v, kc, vc, at)
    q = torch.randn(1, Q, H, D, device=DEV).half()
    order = torch.arange(5, dtype=torch.int32, device=DEV)[None]
    want, _ = check(q, kc, vc, order, lens, "small")

    pages = 2**33 // (4 * H * D * page) + 3
    joint = torch.full((pages, 2, H, page, D), float("nan"), dtype=torch.float16, device=DEV)
    far_k, far_v = joint[:, 0].transpose(1, 2), joint[:, 1].transpose(1, 2)
    border = 2**32 // (4 * H * D * page)
    table = torch.tensor([[pages - 1, border - 1, 0, border, 2 * border, 7]], dtype=torch.int32, device=DEV)
    w4.cache_append(k, v, far_k, far_v, table[0, at // page].long() * page + at % page)
    wide = torch.zeros(1, Q, H + 2, D + 8, dtype=torch.float16, device=DEV)
    wide[:, :, 1:1 + H, 8:] = q
    out = torch.full((1, Q, H + 1, D), 5.0, dtype=torch.float16, device=DEV)
    w4.paged_attention(wide[:, :, 1:1 + H, 8:], far_k, far_v, table, lens, out=out[:, :, :H])
    assert torch.equal(out[:, :, :H], want) and (out[:, :, H] == 5.0).all()


def test_workspace_of_long_pieces_between_guards():
    for B, Q, n in ((1, 70, 5000), (3, 140, 900), (33, 40, 700)):
        q, kc, vc, table, lens = inputs(B, Q, 8, 4, 64, 16, [max(0, n - 37 * b) for b in range(B)], "bf16")
        want = w4.paged_attention(q, kc, vc, table, lens, return_lse=True)
        for fill in (0x00, 0xFF):
            out, lse = torch.empty_like(q), torch.empty_like(want[1])
            a = w4.PagedAttentionArgs()
            a.q, a.k_cache, a.v_cache, a.out, a.lse, a.table, a.lens = (t.data_ptr() for t in (q, kc, vc, out, lse, table, lens))
            a.batch, a.q_len, a.q_heads, a.kv_heads, a.head_dim = B, Q, 8, 4, 64
            a.pages, a.page_size, a.table_width, a.table_stride, a.scale = kc.shape[0], 16, table.shape[1], table.shape[1], 0.125
            for f, t in (("q_stride", q), ("k_stride", kc), ("v_stride", vc), ("out_stride", out)):
                for i in range(3):
                    getattr(a, f)[i] = t.stride(i)
            need = w4.paged_attention_workspace(a)
            buf = torch.full((need + 8192,), 0xA5, dtype=torch.uint8, device=DEV)
            buf[4096:4096 + need] = fill
            a.workspace, a.workspace_bytes = buf.data_ptr() + 4096, need
            assert need > 0 and w4.paged_attention_raw(a, torch.cuda.current_stream().cuda_stream) == w4.OK
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
            assert (buf[:4096] == 0xA5).all() and (buf[4096 + need:] == 0xA5).all()


def test_prompts_of_more_tiles_than_compute_units():
    """Whole tiles where the table holds little more than the prompt, parts of the last ones where it is wide."""
    q, kc, vc, table, lens = inputs(1, 1030, 34, 34, 64, 16, [1030], "bf16")
    wide = torch.full((1, 300), -1, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    check(q, kc, vc, table, lens, "its own keys")
    check(q, kc, vc, wide, lens, "a wide table")
