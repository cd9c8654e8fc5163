"""The angle of rotary_axes over the whole range of positions (MI355X): within
oracle.block_ref.rotary_bound, which allows 2^-22 turns, at every position, for
frequencies up to 1. Pairs (1, 0) and (0, 1) show the cosine and the sine alone, and f16
resolves them where they are small."""
import numpy as np
import pytest
import torch

import bit_quantized_gemm_amd as w4
import oracle.block_ref as ref

from block_helpers import DEV, assert_within, half_bits, normal_bits, to_dev, values_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("power", [8, 16, 23, 24, 25, 27, 29, 31])
def test_positions_up_to(power, interleaved):
    rng = np.random.default_rng(power)
    L, P = 4096, 8
    freq = np.concatenate([[1.0], rng.uniform(0.25, 1.0, P - 1)]).astype(np.float32)
    pos = np.minimum(rng.integers(-2**power, 2**power + 1, size=(1, L, 2)), 2**31 - 1).astype(np.int32)
    pos[0, 0], pos[0, 1], pos[0, 2] = 2**power - 1, -2**power, 0
    xf = np.zeros((1, L, 3, 2 * P))
    first, second = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, P), slice(P, None))
    xf[:, :, 0, first], xf[:, :, 1, second] = 1.0, 1.0
    x = half_bits(xf, "f16")
    x[:, :, 2] = normal_bits(rng, (1, L, 2 * P), "f16")
    for inverse in (False, True):
        y = ref.rotary_ref(x, pos, freq, (3, 5), interleaved, inverse, "f16")
        got = w4.rotary_axes(to_dev(x, "f16"), torch.from_numpy(pos).to(DEV), torch.from_numpy(freq).to(DEV), (3, 5),
                             interleaved=interleaved, inverse=inverse)
        assert_within(values_of(got), y, ref.rotary_bound(x, y, (3, 5), interleaved, "f16"), f"2^{power} inverse={inverse}")


@pytest.mark.parametrize("freq", [16.0, 1e4, 1e-20, 1e-38])
def test_other_frequencies(freq):
    """Above 1 the angle is off by 2^-53 of itself besides (three roundings in float64, one of the oracle's)."""
    rng = np.random.default_rng(3)
    pos = rng.integers(-2**31, 2**31, size=(1, 2048, 1)).astype(np.int32)
    x = normal_bits(rng, (1, 2048, 2, 2), "f16")
    f = np.full(1, freq, dtype=np.float32)
    y = ref.rotary_ref(x, pos, f, (1,), True, False, "f16")
    got = w4.rotary_axes(to_dev(x, "f16"), torch.from_numpy(pos).to(DEV), torch.from_numpy(f).to(DEV), (1,))
    more = np.abs(pos.astype(np.float64) * f[0])[..., None] * 4 * 2.0 ** -53 * 4      # |values| below 4.5, two of them a sum
    assert_within(values_of(got), y, ref.rotary_bound(x, y, (1,), True, "f16") + 2 * more, f"frequency {freq}")
