"""Rows taken again because a value that some of them do not see is no number (MI355X): their weights
still add to one, whatever the scores are. Weights are rounded to the 16-bit type (u = 2^-8
or 2^-11) and their sum is not, so values of one come back within u, 2^-18 for the float32
sums, and half a spacing of the result (u / 2)."""
import numpy as np
import pytest
import torch

import bit_quantized_gemm_amd as w4

from block_helpers import DEV, TORCH, assert_within, values_of

pytestmark = pytest.mark.gpu
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
SIZES = [("bf16", s) for s in (1.0, 1e4, 1e6, 1e8, 1e12)] + [("f16", s) for s in (1.0, 150.0, 3e3)]
NAN = float("nan")


def same_as_one(got, first, dtype, what):
    """Values of one but for NaN in the first place of some keys, the earliest of them key `first`."""
    got = values_of(got)
    assert_within(got[..., 1:], np.ones_like(got[..., 1:]), 1.5 * U[dtype] + 2.0 ** -18, what)
    assert_within(got[:first, :, :1], np.ones_like(got[:first, :, :1]), 1.5 * U[dtype] + 2.0 ** -18, what + " before")
    assert np.isnan(got[first:, :, 0]).all()


@pytest.mark.parametrize("D", [40, 64, 128])
@pytest.mark.parametrize("dtype,size", SIZES)
@pytest.mark.parametrize("wide", [False, True])
def test_packed(wide, dtype, size, D):
    n, HQ, HKV, T = 300, 4, 2, 6000 if wide else 310
    print(f"case: {wide} {dtype} {size} D{D}", flush=True)
    g = torch.Generator().manual_seed(D)
    q, k = (torch.randn(T, h, D, generator=g) * s for h, s in ((HQ, size), (HKV, 1.0)))
    v = torch.ones(T, HKV, D)
    v[10:n:3, :, 0] = NAN
    starts = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    out, lse = w4.packed_attention(*(t.to(TORCH[dtype]).to(DEV) for t in (q, k, v)), starts, scale=1.0, return_lse=True)
    same_as_one(out[:n], 10, dtype, f"{dtype} {size}")
    assert torch.isfinite(lse[:, :n]).all()


@pytest.mark.parametrize("Q", [20, 150])       # the kernel of few rows and of many
@pytest.mark.parametrize("dtype,size", SIZES)
@pytest.mark.parametrize("hole", [False, True])
def test_paged(hole, dtype, size, Q):
    HQ, HKV, D, page, before = 4, 2, 72, 16, 700
    n = Q + before
    print(f"case: {Q} {dtype} {size} {hole}", flush=True)
    g = torch.Generator().manual_seed(Q)
    pages = -(-n // page)
    q = torch.randn(1, Q, HQ, D, generator=g) * size
    kc = torch.randn(pages, page, HKV, D, generator=g)
    vc = torch.ones(pages, page, HKV, D)
    vc.view(-1, HKV, D)[before + 10::3, :, 0] = NAN
    table = torch.arange(pages, dtype=torch.int32)[None]
    if hole:
        table[0, 5] = -1
    out, lse = w4.paged_attention(*(t.to(TORCH[dtype]).to(DEV) for t in (q, kc, vc)), table.to(DEV), torch.tensor([n], dtype=torch.int32, device=DEV),
                                  scale=1.0, return_lse=True)
    same_as_one(out[0], 10, dtype, f"{Q} {dtype} {size}")
    assert torch.isfinite(lse).all()


@pytest.mark.parametrize("wide", [False, True])
def test_result_and_lse_go_together(wide):
    """The weights exp(s - lse) of the keys that a row sees, from its own result: with value j a one in
    place j of the head, out is the weights themselves, which a NaN behind them changes by no more than
    the score's float32 error."""
    T, n, D = 24000 if wide else 70, 64, 64
    g = torch.Generator().manual_seed(3)
    q, k = (torch.randn(T, 1, D, generator=g).bfloat16().to(DEV) for _ in range(2))
    v = torch.zeros(T, 1, D)
    v[:n, 0] = torch.eye(n)
    v = v.bfloat16().to(DEV)
    starts = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    bad = v.clone()
    bad[n - 1, 0, 3] = NAN
    want, got = (w4.packed_attention(q, k, t, starts, return_lse=True) for t in (v, bad))
    rows = slice(0, n - 1)
    # scores below 2^6, each side's off by (D + 8) 2^-24 2^6 < 2^-11; a weight and out are rounded by 2^-8 of them on each side
    assert ((want[0][rows].float() - got[0][rows].float()).abs() <= (2.0 ** -6 + 2.0 ** -9) * want[0][rows].float()).all()
    assert ((want[1][:, rows] - got[1][:, rows]).abs() <= 2.0 ** -10).all()
    assert got[0][n - 1, 0, 3].isnan()
