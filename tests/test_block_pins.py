"""Pins of oracle/block_ref.py (CPU): exact rational arithmetic, closed forms
and planted mistakes, the mistakes in copies of the oracle's inputs."""
from fractions import Fraction

import numpy as np
import pytest

import oracle.block_ref as ref
from oracle.w4a4_ref import dequantize_mx, half_bits_to_f64

from block_helpers import half_bits

GRID = [Fraction(n, 2) for n in (0, 1, 2, 3, 4, 6, 8, 12)]


def _exact_block(values):
    """(scale byte, codes) of 32 finite values by exact search."""
    vs = [Fraction(float(v)) for v in values]
    top = max(abs(v) for v in vs)
    e = -127
    if top > 0:
        e = 0
        while Fraction(2) ** (e + 1) <= top:
            e += 1
        while Fraction(2) ** e > top:
            e -= 1
        e = max(e - 2, -127)
    codes = []
    for raw, v in zip(values, vs):
        a = abs(v) / Fraction(2) ** e
        best = min(range(8), key=lambda c: (abs(GRID[c] - a), c % 2))
        codes.append(best + (8 if np.signbit(raw) else 0))
    return e + 127, codes


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_quantize_against_exact_search(dtype):
    rng = np.random.default_rng(5)
    rows = []
    for i in range(24):
        rows.append(rng.standard_normal(32) * 2.0 ** rng.integers(-20, 12))
    ties = np.tile([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.99], 4) * np.where(np.arange(32) % 3 == 0, -1, 1)
    rows += [ties, ties / 1024, np.zeros(32), -np.zeros(32), np.full(32, 1e-7), np.eye(1, 32, 7)[0] * 4.0]
    bits = half_bits(np.array(rows), dtype)
    bits = np.concatenate([bits, np.arange(32, dtype=np.uint16)[None], 0x8000 + np.arange(32, dtype=np.uint16)[None]])
    act, sc = ref.quantize_mxfp4_ref(bits, dtype)
    vals = half_bits_to_f64(bits, dtype)
    for m in range(len(bits)):
        byte, codes = _exact_block(vals[m])
        assert sc[0, m] == byte, (m, sc[0, m], byte)
        got = np.stack([act[m] & 15, act[m] >> 4], -1).reshape(-1)
        assert got.tolist() == codes, m


def test_quantize_layout_and_special_blocks():
    x = np.zeros((3, 96), dtype=np.float32)
    x[1, 32 + 5] = 8.0            # row 1, block 1: scale 2^1, code 4.0 in an odd position
    x[2, 64] = np.nan
    x[0, 3] = np.inf
    bits = half_bits(x, "bf16")
    act, sc = ref.quantize_mxfp4_ref(bits, "bf16")
    assert sc[:, 1].tolist() == [0, 128, 0] and act[1, (32 + 4) // 2] == 6 << 4
    assert sc[2, 2] == 255 and sc[0, 0] == 255 and not act[2, 32:].any() and not act[0, :16].any()


def test_quantize_round_trip():
    # values already on the grid of a block that holds a 4 or a 6 come back exactly
    rng = np.random.default_rng(6)
    act = rng.integers(0, 256, size=(20, 64), dtype=np.uint8)
    act[:, ::16] = act[:, ::16] & 0xF0 | 6 | (rng.integers(0, 2, size=(20, 4), dtype=np.uint8))
    sc = rng.integers(110, 140, size=(4, 20), dtype=np.uint8)
    v = dequantize_mx(act, sc)
    got, gs = ref.quantize_mxfp4_ref(half_bits(v, "bf16"), "bf16")
    assert np.array_equal(gs, sc) and np.array_equal(got, act)


@pytest.mark.parametrize("interleaved", [True, False])
def test_rotary_closed_forms(interleaved):
    rng = np.random.default_rng(7)
    x = half_bits(rng.standard_normal((2, 3, 2, 12)), "bf16")
    pos = rng.integers(-50, 50, size=(2, 3, 2)).astype(np.int32)
    f = np.array([0.5, 0.25, 2.0, 0.125], dtype=np.float32)
    y = ref.rotary_ref(x, pos, f, (1, 3), interleaved)
    v = half_bits_to_f64(x)
    assert np.array_equal(y[..., 8:], v[..., 8:])                         # past the pairs
    i0, i1 = (2, 3) if interleaved else (1, 5)                            # pair 1 turns by axis 1
    z = (v[..., i0] + 1j * v[..., i1]) * np.exp(1j * pos[..., 1] * 0.25)[..., None]
    assert np.allclose(y[..., i0] + 1j * y[..., i1], z, atol=1e-14)
    # the length of a pair stays; the inverse of the inverse is the map itself
    assert np.allclose((y ** 2).sum(-1), (v ** 2).sum(-1))
    w = ref.rotary_ref(x, -pos, f, (1, 3), interleaved)
    assert np.allclose(w, ref.rotary_ref(x, pos, f, (1, 3), interleaved, inverse=True))


def test_rotary_gradient_is_the_inverse():
    """d(g . y)/dx by differences equals the inverse rotation of g."""
    rng = np.random.default_rng(8)
    pos, f = rng.integers(0, 9, size=(1, 1, 2)).astype(np.int32), np.array([1.0, 0.3, 0.7], dtype=np.float32)
    x, g = rng.integers(-4, 5, size=(1, 1, 1, 8)) * 1.0, rng.integers(-4, 5, size=(1, 1, 1, 8)) * 1.0
    gi = ref.rotary_ref(half_bits(g, "f16"), pos, f, (1, 2), True, inverse=True, dtype="f16")
    for i in range(8):
        d = np.zeros_like(x)
        d[..., i] = 0.5
        hi = (ref.rotary_ref(half_bits(x + d, "f16"), pos, f, (1, 2), dtype="f16") * g).sum()
        lo = (ref.rotary_ref(half_bits(x - d, "f16"), pos, f, (1, 2), dtype="f16") * g).sum()
        assert abs((hi - lo) - gi[0, 0, 0, i]) < 1e-12


def test_attention_brute_force_and_closed_forms():
    rng = np.random.default_rng(9)
    q, k, v = (half_bits(rng.standard_normal(s), "f16") for s in ((2, 2, 4, 8), (2, 5, 2, 8), (2, 5, 2, 8)))
    out, lse, bound, lb = ref.attention_ref(q, k, v, [3, 0], 0.5, "f16")
    qf, kf, vf = (half_bits_to_f64(t, "f16") for t in (q, k, v))
    for i in range(2):
        for h in range(4):
            s = [0.5 * sum(qf[0, i, h, d] * kf[0, j, h // 2, d] for d in range(8)) for j in range(3)]
            w = np.exp(s)
            assert np.allclose(out[0, i, h], (w[:, None] * vf[0, :3, h // 2]).sum(0) / w.sum(), atol=1e-13)
            assert abs(lse[0, h, i] - np.log(w.sum())) < 1e-13
    assert not out[1].any() and np.isneginf(lse[1]).all()
    # one key: its value; equal keys: the mean
    o1 = ref.attention_ref(q, k, v, [1, 1], 0.5, "f16")[0]
    assert np.allclose(o1[0, :, 0], vf[0, 0, 0])
    same = np.repeat(k[:, :1], 5, axis=1)
    o2 = ref.attention_ref(q, same, v, [4, 4], 0.5, "f16")[0]
    assert np.allclose(o2[1, :, 3], vf[1, :4, 1].mean(0))


@pytest.mark.parametrize("mistake", ["transposed scale", "other scale factor", "keys past the length", "head order"])
def test_attention_bound_rejects(mistake):
    """The bound is tight enough that planted mistakes fall outside it."""
    rng = np.random.default_rng(10)
    q, k, v = (half_bits(rng.standard_normal(s), "bf16") for s in ((1, 4, 4, 64), (1, 40, 2, 64), (1, 40, 2, 64)))
    out, lse, bound, lb = ref.attention_ref(q, k, v, [33], 0.125, "bf16")
    args = [q, k, v, [33], 0.125]
    if mistake == "transposed scale":
        args[2] = np.ascontiguousarray(v[..., ::-1])
    elif mistake == "other scale factor":
        args[4] = 0.125 * 1.1
    elif mistake == "keys past the length":
        args[3] = [34]
    else:
        args[0] = np.ascontiguousarray(q[:, :, ::-1])
    wrong = ref.attention_ref(*args, "bf16")[0]
    assert (np.abs(wrong - out) > bound).any()
