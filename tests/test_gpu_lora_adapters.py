"""lora_adapters against the float64 oracle, on every element (MI355X): rows in any order, ranks
of their own, rows without an adapter, odd sizes, strides, in place, streams and graphs."""
import numpy as np
import pytest
import torch

import bit_quantized_gemm_amd as w4
import oracle.request_ref as ref

from block_helpers import DEV, TORCH, assert_within, bits_of, values_of

pytestmark = pytest.mark.gpu


def inputs(M, A, K, N, R, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + M + 3 * N + 7 * K + R)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g) * std).to(TORCH[dtype]).to(DEV)
    y, x, down, up = normal(M, N), normal(M, K), normal(A, R, K, std=K ** -0.5), normal(A, R, N, std=0.5)
    return y, x, down, up, (torch.rand(A, generator=g) + 0.5).to(DEV)


def order(kind, M, A, seed=1):
    rng = np.random.default_rng(seed + M + A)
    ids = {"one": np.zeros(M), "each": np.arange(M) % A, "any": rng.integers(-1, A, M), "none": np.full(M, -1),
           "outside": rng.choice([-2**31, -7, A, A + 5, 2**31 - 1, 0], M),
           "runs": np.sort(rng.integers(0, A, M)), "gaps": np.where(np.arange(M) // 5 % 2 == 0, -1, np.arange(M) // 23 % A)}[kind]
    return torch.from_numpy(ids.astype(np.int32)).to(DEV)


def check(args, adapter, dtype, what, scaling=None, ranks=None, **kw):
    y, x, down, up = args
    v = [values_of(t) for t in args]          # (before an in-place call changes y)
    got = w4.lora_adapters(y, x, down, up, adapter, scaling=scaling, ranks=ranks, **kw)
    want, bound = ref.lora_adapters_ref(*v, adapter.cpu().numpy(), None if scaling is None else scaling.cpu().numpy(),
                                        None if ranks is None else ranks.cpu().numpy(), dtype)
    assert_within(values_of(got), want, bound, what)
    return got


@pytest.mark.parametrize("kind", ["one", "each", "any", "none", "outside", "runs", "gaps"])
@pytest.mark.parametrize("M,A,K,N,R,dtype", [
    (1, 1, 8, 1, 1, "bf16"), (1, 3, 3072, 9216, 16, "f16"), (2, 2, 40, 7, 3, "bf16"), (16, 4, 264, 64, 17, "f16"), (33, 5, 1000, 1001, 33, "bf16"),
    (64, 16, 1032, 520, 32, "bf16"), (65, 70, 128, 200, 64, "f16"), (257, 8, 72, 265, 8, "bf16"), (300, 40, 2056, 333, 128, "f16"),
    (511, 3, 512, 72, 100, "bf16"), (1030, 6, 320, 136, 65, "f16")])
def test_sizes_and_orders(M, A, K, N, R, dtype, kind):
    print(f"case: {M}x{K}->{N} A{A} R{R} {dtype} {kind}", flush=True)
    *args, scaling = inputs(M, A, K, N, R, dtype)
    check(args, order(kind, M, A), dtype, f"{M}x{K}->{N}", scaling=scaling)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N", [(7, 200), (90, 1001), (400, 264)])
def test_ranks_of_their_own(M, N, dtype):
    """Ranks from none to all, past both ends; what lies behind them is NaN."""
    A, K, R = 9, 520, 48
    y, x, down, up, scaling = inputs(M, A, K, N, R, dtype)
    ranks = torch.tensor([0, 1, 15, 16, 17, 33, 48, 99, -3], dtype=torch.int32, device=DEV)
    for a, r in enumerate(ranks.tolist()):
        down[a, max(r, 0):], up[a, max(r, 0):] = float("nan"), float("nan")
    want = w4.lora_adapters(y, x, down.nan_to_num(0), up.nan_to_num(0), order("any", M, A), scaling=scaling)
    got = w4.lora_adapters(y, x, down, up, order("any", M, A), scaling=scaling, ranks=ranks)
    assert torch.equal(got, want)
    zero = [t.nan_to_num(0) for t in (down, up)]
    check((y, x, *zero), order("any", M, A), dtype, "ranks", scaling=scaling, ranks=ranks)
    check((y, x, *zero), order("runs", M, A), dtype, "no scaling", ranks=ranks)


def test_rows_keep_to_themselves():
    """An infinity or a NaN in a row, or in an adapter, goes to no other row."""
    M, A, K, N, R = 200, 6, 264, 392, 24
    for dtype in ("bf16", "f16"):
        y, x, down, up, scaling = inputs(M, A, K, N, R, dtype)
        ids = order("any", M, A)
        want = w4.lora_adapters(y, x, down, up, ids, scaling=scaling)
        x[3, 5], x[77, 263], y[9, 0] = float("nan"), float("inf"), float("nan")
        down[2, 23, 0], up[4, 0, 391] = float("nan"), float("inf")
        got = w4.lora_adapters(y, x, down, up, ids, scaling=scaling)
        touched = torch.zeros(M, dtype=torch.bool, device=DEV)
        touched[[3, 77, 9]] = True
        clean = ~(touched | (ids == 2) | (ids == 4))
        assert torch.equal(got[clean], want[clean])
        assert got[9, 0].isnan() and torch.equal(got[9, 1:], want[9, 1:]) or ids[9] in (2, 4)
        rest = (ids == 4) & ~touched
        assert torch.equal(got[rest][:, :391], want[rest][:, :391]) and not torch.isfinite(got[rest][:, 391]).any()
        assert got[(ids == 2) & ~touched].isnan().all()


def test_binary16_past_its_range():
    """x @ down^T past 65504, and rows of tiny values: the product with up brings them back."""
    M, A, K, N, R = 40, 2, 512, 136, 20
    y, x, down, up, _ = inputs(M, A, K, N, R, "f16")
    x[::2] *= 2000.0
    down[0] *= 500.0
    up[0] *= 2.0 ** -16
    x[1::4] *= 2.0 ** -8
    down[1] *= 2.0 ** -5
    y *= 2.0 ** -4
    low = values_of(x) @ values_of(down[0]).T
    assert np.abs(low).max() > 1e6
    check((y, x, down, up), order("each", M, A), "f16", "range")


@pytest.mark.parametrize("M,N", [(5, 1001), (64, 512), (300, 77)])
def test_strides_and_in_place(M, N):
    A, K, R = 4, 136, 19
    *args, scaling = inputs(M, A, K, N, R, "bf16")
    y, x, down, up = args
    wide = torch.full((M, N + 13), 5.0, dtype=torch.bfloat16, device=DEV)
    wx = torch.randn(M, 2 * K, device=DEV).bfloat16()
    view, vx = wide[:, 6:6 + N], wx[:, K:]
    view.copy_(y), vx.copy_(x)
    ids = order("any", M, A)
    want = check(args, ids, "bf16", "dense", scaling=scaling)
    assert torch.equal(w4.lora_adapters(view, vx, down, up, ids, scaling=scaling), want)
    got = w4.lora_adapters(view, vx, down, up, ids, scaling=scaling, out=view)
    assert got.data_ptr() == view.data_ptr() and torch.equal(view, want)
    view.fill_(5.0)
    assert (wide == 5.0).all()
    w4.lora_adapters(y, vx, down, up, ids, scaling=scaling, out=view)
    assert torch.equal(view, want)
    view.fill_(5.0)
    assert (wide == 5.0).all()


def test_workspace_between_guards():
    """The C entry point with a workspace of the stated size, holding anything; nothing around it changes."""
    for M, K, N, R in ((1, 3072, 264, 16), (64, 2056, 200, 20), (300, 520, 1001, 33)):
        y, x, down, up, scaling = inputs(M, 5, K, N, R, "bf16")
        ids = order("any", M, 5)
        want = w4.lora_adapters(y, x, down, up, ids, scaling=scaling)
        for fill in (0x00, 0xFF, 0x5A):
            out = torch.empty_like(y)
            a = w4.LoraAdaptersArgs(x.data_ptr(), y.data_ptr(), down.data_ptr(), up.data_ptr(), out.data_ptr(), ids.data_ptr(),
                                    scaling.data_ptr(), 0, M, K, N, 5, R, K, N, N, 0)
            need = w4.lora_adapters_workspace(a)
            buf = torch.full((need + 8192,), 0xA5, dtype=torch.uint8, device=DEV)
            buf[4096:4096 + need] = fill
            a.workspace, a.workspace_bytes = buf.data_ptr() + 4096, need
            assert w4.lora_adapters_raw(a, torch.cuda.current_stream().cuda_stream) == w4.OK
            assert torch.equal(out, want) and (buf[:4096] == 0xA5).all() and (buf[4096 + need:] == 0xA5).all()


def test_streams_and_graph():
    M, A, K, N, R = 70, 6, 520, 648, 32
    *args, scaling = inputs(M, A, K, N, R, "bf16")
    ids = order("any", M, A)
    want = check(args, ids, "bf16", "eager", scaling=scaling)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [w4.lora_adapters(*args, ids, scaling=scaling, stream=s) for s in (side, side.cuda_stream)]
    here = w4.lora_adapters(*args, ids, scaling=scaling)          # at the same time on another stream
    side.synchronize()
    assert all(torch.equal(g, want) for g in got) and torch.equal(here, want)
    held = [t.clone() for t in args]
    hid = ids.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = w4.lora_adapters(*held, hid, scaling=scaling)
    for i in range(4):
        hid.copy_(order("runs" if i % 2 else "any", M, A, seed=i))
        held[1].copy_(args[1] * (i + 1))
        g.replay()
        eager = w4.lora_adapters(args[0], args[1] * (i + 1), *args[2:], hid, scaling=scaling)
        torch.cuda.synchronize()
        assert torch.equal(kept, eager)


def test_many_rows_and_adapters():
    """More adapters than a tile has rows, thousands of rows, weights past 2^31 bytes."""
    M, A, K, N, R = 4352, 600, 3072, 256, 16
    y, x = (torch.randn(M, n, device=DEV).bfloat16() for n in (N, K))
    down = torch.empty(A, 128, K, device=DEV, dtype=torch.bfloat16).normal_(std=0.02)       # 472 MB
    up = torch.empty(A, 128, N, device=DEV, dtype=torch.bfloat16).normal_(std=0.5)
    ids = torch.randint(-1, A, (M,), device=DEV, dtype=torch.int32)
    ranks = torch.full((A,), R, dtype=torch.int32, device=DEV)
    got = w4.lora_adapters(y, x, down, up, ids, ranks=ranks)
    pick = torch.randperm(M)[:200].tolist() + [0, M - 1]
    use = [a for a in ids[pick].tolist()]
    t = [values_of(v) for v in (y[pick], x[pick], torch.stack([down[max(a, 0), :R] for a in use]), torch.stack([up[max(a, 0), :R] for a in use]))]
    want, bound = ref.lora_adapters_ref(*t, [i if a >= 0 else -1 for i, a in enumerate(use)], dtype="bf16")
    assert_within(values_of(got[pick]), want, bound, "picked rows")
    big = torch.zeros(3, 128, 2**23, device=DEV, dtype=torch.bfloat16)                     # adapters 2 GiB apart
    big[2, 5, -64:] = 1.0
    one = torch.zeros(4, 2**23, device=DEV, dtype=torch.bfloat16)
    one[:, -64:] = 1.0
    last = torch.tensor([2, 0, 2, 1], dtype=torch.int32, device=DEV)
    out = w4.lora_adapters(torch.zeros(4, 16, device=DEV, dtype=torch.bfloat16), one, big, torch.ones(3, 128, 16, device=DEV, dtype=torch.bfloat16), last)
    assert out[:, 0].tolist() == [64.0, 0.0, 64.0, 0.0] and bits_of(out).shape == (4, 16)


@pytest.mark.parametrize("M,A,K,N,R,dtype", [
    (20000, 7, 64, 256, 16, "bf16"),        # more rows than the grouping holds in registers
    (700, 5000, 72, 8200, 9, "f16"),        # more adapters than it takes
    (3000, 4096, 40, 1500, 3, "bf16"),      # as many as it takes, most with a row or none
    (1500, 3, 520, 1001, 128, "f16"), (9000, 2, 8, 503, 33, "bf16")])
def test_many_rows(M, A, K, N, R, dtype):
    """Picked rows against the oracle, the same bytes each time, in place, and replayed from a graph."""
    y, x, down, up, scaling = inputs(M, A, K, N, R, dtype)
    ids = order("any", M, A)
    first = w4.lora_adapters(y, x, down, up, ids, scaling=scaling)
    pick = np.random.default_rng(M).permutation(M)[:150].tolist() + [0, M - 1]
    use = ids[pick].tolist()
    t = [values_of(v) for v in (y[pick], x[pick], torch.stack([down[max(a, 0)] for a in use]), torch.stack([up[max(a, 0)] for a in use]))]
    s = np.array([float(scaling[max(a, 0)]) for a in use], dtype=np.float32)
    want, bound = ref.lora_adapters_ref(*t, [i if a >= 0 else -1 for i, a in enumerate(use)], s, dtype=dtype)
    assert_within(values_of(first[pick]), want, bound, f"{M} rows of {A}")
    assert torch.equal(first[ids < 0], y[ids < 0])
    for _ in range(3):
        assert torch.equal(w4.lora_adapters(y, x, down, up, ids, scaling=scaling), first)
    held, hid = y.clone(), ids.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = w4.lora_adapters(held, x, down, up, hid, scaling=scaling, out=held)
    for i in range(3):
        held.copy_(y)
        hid.copy_(ids.roll(i))
        g.replay()
        eager = w4.lora_adapters(y, x, down, up, ids.roll(i), scaling=scaling)
        torch.cuda.synchronize()
        assert torch.equal(kept, eager)
