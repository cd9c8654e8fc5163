"""cross_attention where scores are large (MI355X): a float32 score past 2^24 has no
fraction left, so that what is held here is what stays true whatever its rounding is.
Weights are rounded to the 16-bit type (u = 2^-8 or 2^-11) and their sum is not, so equal
values come back within u, 2^-18 for the float32 sums, and half a spacing of the
result."""
import numpy as np
import pytest
import torch

import bit_quantized_gemm_amd as w4
import oracle.block_ref as ref
from oracle.w4a4_ref import half_bits_to_f64

from block_helpers import DEV, assert_within, half_bits, normal_bits, to_dev, values_of

pytestmark = pytest.mark.gpu
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
# (LQ, LK): the few-row kernel, its cut keys, the 128-row one, its cut keys
SIZES = [(1, 1), (3, 40), (2, 3000), (129, 1), (200, 100), (130, 1500)]


def run(q, k, v, dtype, lens=None):
    out, lse = w4.cross_attention(*(to_dev(t, dtype) for t in (q, k, v)), return_lse=True,
                                  kv_lens=None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV))
    return values_of(out), lse.double().cpu().numpy()


@pytest.mark.parametrize("dtype,size", [("f16", s) for s in (100.0, 1500.0, 2500.0, 4000.0, 30000.0, 60000.0)] +
                         [("bf16", s) for s in (2500.0, 1e5, 1e6, 1e10, 1e16)])
@pytest.mark.parametrize("LQ,LK", SIZES)
def test_equal_scores(LQ, LK, dtype, size):
    """All scores alike: the mean of the values, the value itself for one key."""
    print(f"case: {LQ}x{LK} {dtype} {size}", flush=True)
    rng = np.random.default_rng(LQ + LK)
    D = 128
    q, k = (half_bits(np.full((2, n, 1, D), size), dtype) for n in (LQ, LK))
    v = normal_bits(rng, (2, LK, 1, D), dtype)
    out, lse = run(q, k, v, dtype)
    vv = half_bits_to_f64(v, dtype)[:, :, 0]
    want = np.broadcast_to(vv.mean(1)[:, None, None], out.shape)
    bound = np.abs(vv).mean(1)[:, None, None] * (U[dtype] + 2.0 ** -18) + 0.5 * ref.half_spacing(want, dtype) * (1 + 2.0 ** -6)
    assert_within(out, want, bound, "mean")
    s = float(half_bits_to_f64(q, dtype).flat[0]) ** 2 * D ** 0.5
    assert (np.abs(lse - (s + np.log(LK))) <= 2.0 ** -20 * (s + 10)).all()


@pytest.mark.parametrize("dtype,size", [("f16", s) for s in (30.0, 300.0, 1000.0, 3000.0, 8000.0, 15000.0)] +
                         [("bf16", s) for s in (300.0, 3000.0, 1e5, 1e7, 1e12)])
@pytest.mark.parametrize("LQ,LK", SIZES)
def test_weights_add_to_one(LQ, LK, dtype, size):
    """Values of one give one, whatever the scores; where the largest score leads by more
    than the scores' own rounding, the result is its value, as one of equal values. (Rows
    that an infinity among the 16-bit inputs reaches are left out.)"""
    print(f"case: {LQ}x{LK} {dtype} {size}", flush=True)
    rng = np.random.default_rng(LQ + LK)
    D = 64
    q, k = (normal_bits(rng, (2, n, 2, D), dtype, size) for n in (LQ, LK))
    lens = [LK, max(1, LK - LK // 3)]
    ones, lse = run(q, k, half_bits(np.ones((2, LK, 2, D)), dtype), dtype, lens)
    v = normal_bits(rng, (2, LK, 2, D), dtype)
    out, _ = run(q, k, v, dtype, lens)
    qf, kf, vf = (half_bits_to_f64(t, dtype) for t in (q, k, v))
    clear = 0
    for b in range(2):
        for h in range(2):
            with np.errstate(invalid="ignore"):
                s = qf[b, :, h] @ kf[b, :lens[b], h].T / 8
                noise = (np.abs(qf[b, :, h]) @ np.abs(kf[b, :lens[b], h]).T).max(1) / 8 * (D + 8) * 2.0 ** -23
                best = s.argmax(1)
                second = np.where(np.arange(s.shape[1])[None] == best[:, None], -np.inf, s).max(1)
                fine = np.isfinite(s).all(1)
                rows = fine & (s.max(1) - second > noise + 40)
            assert_within(ones[b, fine, h], np.ones((fine.sum(), D)), U[dtype] * 1.5 + 2.0 ** -18, "ones")
            assert np.isfinite(lse[b, h, fine]).all()
            want = vf[b, best[rows], h]
            assert_within(out[b, rows, h], want, np.abs(want) * (U[dtype] + 2.0 ** -18) +
                          0.5 * ref.half_spacing(want, dtype) * (1 + 2.0 ** -6), "one weight")
            clear += int(rows.sum())
    print(f"  rows with one weight: {clear}", flush=True)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("LQ", [1, 140])
@pytest.mark.parametrize("top", [22, 24, 25, 26, 27, 28, 29, 30])
def test_maximum_that_rises_by_little(LQ, top, dtype):
    """Scores near 2^top (in powers of two) that rise along the keys by a few units in
    their last place: neighbouring tiles differ by less, and by more, than the growth at
    which sums are rescaled. Values of one give one."""
    print(f"case: {LQ} 2^{top} {dtype}", flush=True)
    D, LK = 64, 500
    rng = np.random.default_rng(top)
    base = (2.0 ** top * np.log(2) * 8 / D) ** 0.5
    q = half_bits(np.full((1, LQ, 1, D), base), dtype)
    kf = half_bits_to_f64(half_bits(np.full((1, LK, 1, D), base), dtype), dtype)
    kf[..., 0] = np.linspace(0, 1, LK)[None, :, None] * base        # scores rise by 1/64 over all keys
    kf[..., 1] += rng.uniform(-1, 1, (1, LK, 1)) * base * 2.0 ** -6
    out, lse = run(q, half_bits(kf, dtype), half_bits(np.ones((1, LK, 1, D)), dtype), dtype)
    assert_within(out, np.ones_like(out), U[dtype] * 1.5 + 2.0 ** -18, "ones")
    assert np.isfinite(lse).all()
