"""lora_adapters on rows grouped by adapter, the way of many rows (MI355X): against the float64 oracle on
every element, in every order, with ranks of their own, strides, in place, values that are no numbers and
workspaces that hold anything. Each case says by its workspace that it is grouped."""
import numpy as np
import pytest
import torch

import bit_quantized_gemm_amd as w4
import oracle.request_ref as ref

from block_helpers import DEV, TORCH, assert_within, values_of
from test_gpu_lora_adapters import check, inputs, order

pytestmark = pytest.mark.gpu


def is_grouped(M, A, K, N, R, dtype):
    """Few rows keep whole slices of float32 sums in the workspace; groups need more beside these."""
    def need(columns):
        return w4.lora_adapters_workspace(w4.LoraAdaptersArgs(rows=M, K=K, N=columns, adapters=A, rank=R, f16=dtype == "f16"))
    sums = M * 4 * next(p for p in (16, 32, 64, 128) if p >= R)
    assert need(1) % sums == 0
    return need(N) % sums != 0


SIZES = [(4200, 5, 136, 1001, 9, "bf16"), (4200, 4, 8, 1001, 16, "f16"), (2100, 8, 264, 1001, 32, "bf16"), (2100, 8, 72, 1003, 17, "f16"),
         (4200, 6, 520, 264, 48, "bf16"), (1100, 40, 1000, 960, 64, "f16"), (1700, 3, 72, 320, 100, "bf16"), (530, 300, 2056, 1000, 65, "f16")]


@pytest.mark.parametrize("kind", ["one", "each", "any", "outside", "runs", "gaps"])
@pytest.mark.parametrize("M,A,K,N,R,dtype", SIZES)
def test_sizes_and_orders(M, A, K, N, R, dtype, kind):
    print(f"case: {M}x{K}->{N} A{A} R{R} {dtype} {kind}", flush=True)
    assert is_grouped(M, A, K, N, R, dtype)
    *args, scaling = inputs(M, A, K, N, R, dtype)
    check(args, order(kind, M, A), dtype, f"{M}x{K}->{N}", scaling=scaling)


@pytest.mark.parametrize("N,dtype", [(7, "bf16"), (3, "f16"), (5, "f16")])
def test_fewer_columns_than_an_access(N, dtype):
    M, A, K, R = -(-2**26 // (128 * N)) + 61, 3, 8, 100
    assert is_grouped(M, A, K, N, R, dtype)
    y, x, down, up, scaling = inputs(M, A, K, N, R, dtype)
    ids = order("any", M, A)
    got = w4.lora_adapters(y, x, down, up, ids, scaling=scaling)
    pick = np.sort(np.random.default_rng(N).permutation(M)[:3000]).tolist()
    t = [values_of(v) for v in (y[pick], x[pick], down, up)]
    want, bound = ref.lora_adapters_ref(*t, ids.cpu().numpy()[pick], scaling.cpu().numpy(), dtype=dtype)
    assert_within(values_of(got[pick]), want, bound, f"{N} columns")
    assert torch.equal(got[ids < 0], y[ids < 0])


def test_none_of_many():
    M, A, K, N, R = 4200, 5, 136, 1001, 9
    *args, scaling = inputs(M, A, K, N, R, "bf16")
    assert is_grouped(M, A, K, N, R, "bf16")
    got = w4.lora_adapters(*args, order("none", M, A), scaling=scaling)
    assert torch.equal(got, args[0])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_ranks_of_their_own(dtype):
    """Ranks from none to all, past both ends, behind which there is NaN; the workspace, of the stated
    size between guards, holds NaN, so that nothing of a row is taken that its own rank does not write."""
    M, A, K, N, R = 4200, 9, 520, 264, 48
    assert is_grouped(M, A, K, N, R, dtype)
    y, x, down, up, scaling = inputs(M, A, K, N, R, dtype)
    ranks = torch.tensor([0, 1, 15, 16, 17, 33, 48, 99, -3], dtype=torch.int32, device=DEV)
    for a, r in enumerate(ranks.tolist()):
        down[a, max(r, 0):], up[a, max(r, 0):] = float("nan"), float("nan")
    zero = [t.nan_to_num(0) for t in (down, up)]
    for kind in ("any", "runs"):
        ids = order(kind, M, A)
        want = check((y, x, *zero), ids, dtype, f"ranks {kind}", scaling=scaling, ranks=ranks)
        for fill in (0xFF, 0x00, 0x5A):
            out = torch.empty_like(y)
            a = w4.LoraAdaptersArgs(x.data_ptr(), y.data_ptr(), down.data_ptr(), up.data_ptr(), out.data_ptr(), ids.data_ptr(),
                                    scaling.data_ptr(), ranks.data_ptr(), M, K, N, A, R, K, N, N, dtype == "f16")
            need = w4.lora_adapters_workspace(a)
            buf = torch.full((need + 8192,), 0xA5, dtype=torch.uint8, device=DEV)
            buf[4096:4096 + need] = fill
            a.workspace, a.workspace_bytes = buf.data_ptr() + 4096, need
            assert w4.lora_adapters_raw(a, torch.cuda.current_stream().cuda_stream) == w4.OK
            assert torch.equal(out, want) and (buf[:4096] == 0xA5).all() and (buf[4096 + need:] == 0xA5).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_rows_keep_to_themselves(dtype):
    """An infinity or a NaN in a row, or in an adapter, goes to no other row."""
    M, A, K, N, R = 2200, 6, 264, 1001, 24
    assert is_grouped(M, A, K, N, R, dtype)
    y, x, down, up, scaling = inputs(M, A, K, N, R, dtype)
    ids = order("any", M, A)
    want = w4.lora_adapters(y, x, down, up, ids, scaling=scaling)
    x[3, 5], x[777, 263], y[9, 0] = float("nan"), float("inf"), float("nan")
    down[2, 23, 0], up[4, 0, 1000] = float("nan"), float("inf")
    got = w4.lora_adapters(y, x, down, up, ids, scaling=scaling)
    touched = torch.zeros(M, dtype=torch.bool, device=DEV)
    touched[[3, 777, 9]] = True
    clean = ~(touched | (ids == 2) | (ids == 4))
    assert torch.equal(got[clean], want[clean])
    assert got[9, 0].isnan() and (torch.equal(got[9, 1:], want[9, 1:]) or ids[9] in (2, 4))
    rest = (ids == 4) & ~touched
    assert torch.equal(got[rest][:, :1000], want[rest][:, :1000]) and not torch.isfinite(got[rest][:, 1000]).any()
    assert got[(ids == 2) & ~touched].isnan().all()


def test_binary16_past_its_range():
    """x @ down^T past 65504, and rows of tiny values, with ranks of their own."""
    M, A, K, N, R = 4200, 2, 512, 264, 50
    assert is_grouped(M, A, K, N, R, "f16")
    y, x, down, up, _ = inputs(M, A, K, N, R, "f16")
    x[::2] *= 2000.0
    down[0] *= 500.0
    up[0] *= 2.0 ** -16
    x[1::4] *= 2.0 ** -8
    down[1] *= 2.0 ** -5
    y *= 2.0 ** -4
    low = values_of(x[::2]) @ values_of(down[0]).T
    assert np.abs(low).max() > 1e6
    check((y, x, down, up), order("each", M, A), "f16", "range")
    check((y, x, down, up), order("each", M, A), "f16", "range", ranks=torch.tensor([50, 7], dtype=torch.int32, device=DEV))


@pytest.mark.parametrize("M,N,dtype", [(2200, 1001, "bf16"), (2200, 1000, "f16"), (4300, 515, "f16")])
def test_strides_and_in_place(M, N, dtype):
    A, K, R = 4, 136, 19
    assert is_grouped(M, A, K, N, R, dtype)
    *args, scaling = inputs(M, A, K, N, R, dtype)
    y, x, down, up = args
    wide = torch.full((M, N + 13), 5.0, dtype=TORCH[dtype], device=DEV)
    wx = torch.randn(M, 2 * K, device=DEV).to(TORCH[dtype])
    view, vx = wide[:, 6:6 + N], wx[:, K:]
    view.copy_(y), vx.copy_(x)
    ids = order("any", M, A)
    want = check(args, ids, dtype, "dense", scaling=scaling)
    assert torch.equal(w4.lora_adapters(view, vx, down, up, ids, scaling=scaling), want)
    got = w4.lora_adapters(view, vx, down, up, ids, scaling=scaling, out=view)
    assert got.data_ptr() == view.data_ptr() and torch.equal(view, want)
    view.fill_(5.0)
    assert (wide == 5.0).all()
    w4.lora_adapters(y, vx, down, up, ids, scaling=scaling, out=view)
    assert torch.equal(view, want)
    view.fill_(5.0)
    assert (wide == 5.0).all()


def test_two_streams_at_once_and_replays():
    M, A, K, N, R = 2200, 6, 264, 1001, 24
    *args, scaling = inputs(M, A, K, N, R, "bf16")
    assert is_grouped(M, A, K, N, R, "bf16")
    ids = order("any", M, A)
    want = check(args, ids, "bf16", "eager", scaling=scaling)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(4):
        got += [w4.lora_adapters(*args, ids, scaling=scaling, stream=s) for s in (side, None)]
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
    hid = ids.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = w4.lora_adapters(*args, hid, scaling=scaling)
        again = w4.lora_adapters(kept, *args[1:], hid, scaling=scaling)      # a second call's workspace in the same graph
    for i in range(4):
        hid.copy_(order("runs" if i % 2 else "any", M, A, seed=i))
        g.replay()
        first = w4.lora_adapters(*args, hid, scaling=scaling)
        eager = w4.lora_adapters(first, *args[1:], hid, scaling=scaling)
        torch.cuda.synchronize()
        assert torch.equal(kept, first) and torch.equal(again, eager)
