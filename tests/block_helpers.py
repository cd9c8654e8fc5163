"""Bit patterns on the host, tensors on the device, for the tests of the
operators around the 4-bit layers."""
import numpy as np
import torch

from oracle.w4a4_ref import half_bits_to_f64

DEV = "cuda:0"
TORCH = {"bf16": torch.bfloat16, "f16": torch.float16}


def half_bits(x, dtype):
    """float array -> 16-bit patterns, nearest even."""
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(TORCH[dtype])
    return t.view(torch.int16).numpy().view(np.uint16)


def normal_bits(rng, shape, dtype, std=1.0):
    return half_bits(rng.standard_normal(size=shape) * std, dtype)


def to_dev(bits, dtype):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(TORCH[dtype]).to(DEV)


def bits_of(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def values_of(t):
    return half_bits_to_f64(bits_of(t), "f16" if t.dtype == torch.float16 else "bf16")


def assert_within(got, want, bound, what):
    """|got - want| <= bound everywhere (values, float64)."""
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.array_equal(np.isnan(got), np.isnan(want)), (what, "NaN in other places")
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), (what, "infinities differ")
    ok = np.isfinite(want)
    err = np.abs(got[ok] - want[ok])
    ratio = err / np.maximum(np.broadcast_to(bound, want.shape)[ok], 1e-300)
    worst = float(ratio.max()) if ratio.size else 0.0
    print(f"  {what}: {want.size} values, max err/bound {worst:.3g}", flush=True)
    assert worst <= 1.0 or float(err.max()) == 0.0, (what, worst)
