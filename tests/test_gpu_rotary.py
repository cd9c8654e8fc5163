"""Parity of rotary_axes with the float64 oracle (MI355X) within
oracle.block_ref.rotary_bound; the gradient against the oracle's inverse."""
import numpy as np
import pytest
import torch

import bit_quantized_gemm_amd as w4
import oracle.block_ref as ref

from block_helpers import DEV, assert_within, bits_of, normal_bits, to_dev, values_of

pytestmark = pytest.mark.gpu


def freqs(sections):
    return np.concatenate([10000.0 ** (-np.arange(n) / max(n, 1)) for n in sections]).astype(np.float32)


def call(x, pos, sections, **kw):
    return w4.rotary_axes(x, torch.from_numpy(pos).to(DEV), torch.from_numpy(freqs(sections)).to(DEV), sections, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("B,L,H,D,sections", [
    (1, 1, 1, 2, (1,)), (1, 1, 1, 8, (0, 0, 0)), (2, 3, 1, 10, (2, 1, 2)), (1, 7, 3, 64, (16, 16)),
    (2, 33, 24, 128, (8, 28, 28)), (3, 5, 9, 72, (4, 11, 17)), (8, 1, 9, 72, (4, 11, 17)), (1, 100, 48, 128, (64,)),
    (1, 11, 2, 256, (32, 32, 32, 32)), (2, 9, 300, 16, (3, 0, 5)), (1, 257, 5, 96, (1, 2, 3)), (1, 5, 1, 6, (0, 1))])
def test_sizes(B, L, H, D, sections, interleaved, dtype):
    print(f"case: {B} {L} {H} {D} {sections} {interleaved} {dtype}", flush=True)
    rng = np.random.default_rng(B + L + H + D)
    x = normal_bits(rng, (B, L, H, D), dtype)
    pos = rng.integers(-300, 5000, size=(B, L, len(sections))).astype(np.int32)
    for inverse in (False, True):
        y = ref.rotary_ref(x, pos, freqs(sections), sections, interleaved, inverse, dtype)
        got = call(to_dev(x, dtype), pos, sections, interleaved=interleaved, inverse=inverse)
        assert_within(values_of(got), y, ref.rotary_bound(x, y, sections, interleaved, dtype), f"inverse={inverse}")


@pytest.mark.parametrize("interleaved", [True, False])
def test_large_positions(interleaved):
    """Angles of many turns keep their accuracy, at positions no float32 holds too."""
    rng = np.random.default_rng(1)
    sections = (5, 7, 4)
    x = normal_bits(rng, (1, 40, 2, 32), "f16")
    pos = rng.integers(-2**31, 2**31, size=(1, 40, 3)).astype(np.int32)
    pos[0, 0], pos[0, 1], pos[0, 2] = 2**31 - 1, -2**31, 2**24 + 1
    # at these positions a turn of a pair is exact only as far as float32 of
    # inv_freq / (2 pi) carried in two parts: 2^31 positions x 2^-48 turns
    y = ref.rotary_ref(x, pos, freqs(sections), sections, interleaved, False, "f16")
    bound = ref.rotary_bound(x, y, sections, interleaved, "f16") * (1 + 2.0 ** -6) + 8 * 2.0 ** (31 - 46)
    assert_within(values_of(call(to_dev(x, "f16"), pos, sections, interleaved=interleaved)), y, bound, "large positions")


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("offset", [0, 1, 2, 4])
def test_strided_in_place_and_guard(interleaved, offset):
    """The q and k heads of a joint projection rotated where they are, at addresses of
    every alignment, positions shared by the batch; the v heads and the memory
    around stay."""
    if interleaved and offset == 1:
        offset = 6
    rng = np.random.default_rng(2)
    sections, L = (2, 3, 3), 6
    bits = normal_bits(rng, (2, L, 9, 20), "bf16")
    buf = torch.zeros(bits.size + 64, dtype=torch.bfloat16, device=DEV)
    joint = buf[offset:offset + bits.size].view(bits.shape)
    joint.copy_(to_dev(bits, "bf16"))
    pos = rng.integers(0, 64, size=(L, 3)).astype(np.int32)
    part = joint[:, :, :6]
    out = call(part, pos, sections, interleaved=interleaved, out=part)
    assert out.data_ptr() == part.data_ptr()
    x = np.ascontiguousarray(bits[:, :, :6])
    y = ref.rotary_ref(x, np.broadcast_to(pos, (2, L, 3)), freqs(sections), sections, interleaved)
    assert_within(values_of(part), y, ref.rotary_bound(x, y, sections, interleaved, "bf16"), "in place")
    assert np.array_equal(bits_of(joint[:, :, 6:]), bits[:, :, 6:])
    assert not buf[:offset].any() and not buf[offset + bits.size:].any()


def test_transposed_orders():
    """Heads before tokens in memory, in and out; positions with a stride."""
    rng = np.random.default_rng(3)
    sections = (4, 4)
    x = normal_bits(rng, (2, 5, 7, 24), "f16")
    pos = rng.integers(0, 64, size=(2, 5, 2)).astype(np.int32)
    xt = to_dev(x, "f16").transpose(1, 2).contiguous().transpose(1, 2)
    out = torch.empty(2, 7, 5, 24, dtype=torch.float16, device=DEV).transpose(1, 2)
    wide = torch.zeros(2, 5, 6, dtype=torch.int32, device=DEV)
    wide[..., :2] = torch.from_numpy(pos).to(DEV)
    got = w4.rotary_axes(xt, wide[..., :2], torch.from_numpy(freqs(sections)).to(DEV), sections, out=out)
    y = ref.rotary_ref(x, pos, freqs(sections), sections, dtype="f16")
    assert_within(values_of(got), y, ref.rotary_bound(x, y, sections, True, "f16"), "transposed")


@pytest.mark.parametrize("interleaved", [True, False])
def test_special_values_stay_in_their_pair(interleaved):
    rng = np.random.default_rng(4)
    x = normal_bits(rng, (1, 4, 2, 24), "bf16")
    x[0, 1, 0, 3], x[0, 2, 1, 23] = 0x7FC0, 0x7F81       # a NaN in a pair, a signalling one in the copied part
    pos = np.arange(8, dtype=np.int32).reshape(1, 4, 2)
    got = bits_of(call(to_dev(x, "bf16"), pos, (4, 4), interleaved=interleaved))
    nan = np.isnan(values_of(to_dev(got, "bf16")))
    want = np.zeros_like(nan)
    want[0, 1, 0, [2, 3] if interleaved else [3, 11]] = True
    want[0, 2, 1, 23] = True
    assert np.array_equal(nan, want) and np.array_equal(got[..., 16:], x[..., 16:])


def test_gradient_round_trip_and_empty():
    """The gradient of x is the inverse rotation of the gradient of y; empty tensors do nothing."""
    rng = np.random.default_rng(5)
    sections = (3, 2, 5)
    g = normal_bits(rng, (2, 6, 3, 20), "f16")
    pos = rng.integers(0, 99, size=(2, 6, 3)).astype(np.int32)
    want = ref.rotary_ref(g, pos, freqs(sections), sections, True, True, "f16")
    got = call(to_dev(g, "f16"), pos, sections, inverse=True)
    assert_within(values_of(got), want, ref.rotary_bound(g, want, sections, True, "f16"), "gradient")
    for shape in ((0, 6, 3, 20), (2, 0, 3, 20), (2, 6, 0, 20)):
        x = torch.empty(shape, dtype=torch.float16, device=DEV)
        p = torch.zeros(shape[:2] + (3,), dtype=torch.int32, device=DEV)
        assert w4.rotary_axes(x, p, torch.ones(10, device=DEV), sections).shape == x.shape
