"""Parity of gemm_mxfp4_few with the MXFP4 oracle (MI355X), within the bound of
gemm_mxfp4's tests: 4e-3 T + 1 ulp on every element."""
import numpy as np
import pytest
import torch

import bit_quantized_gemm_amd as w4
import synthetic

from gpu_helpers import ARGS, DEV, assert_parity, full_reference, to_device

pytestmark = pytest.mark.gpu


def run(x, out=None, **kw):
    d = to_device(x)
    y = w4.gemm_mxfp4_few(*(d[k] for k in ARGS), out=out, dtype=torch.float16 if x["dtype"] == "f16" else torch.bfloat16, **kw)
    torch.cuda.synchronize()
    return y


def bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K,R", [
    (1, 1, 32, 0), (1, 16, 32, 1), (1, 3072, 3072, 32), (2, 17, 64, 3), (3, 100, 96, 8), (7, 33, 160, 33),
    (15, 31, 128, 16), (16, 256, 1024, 32), (17, 250, 1056, 128), (32, 1001, 480, 17), (33, 64, 2080, 300),
    (48, 130, 12288, 128), (61, 1001, 3104, 17), (63, 15, 4096, 1024), (64, 512, 512, 0), (64, 48, 32, 40)])
def test_sizes(M, N, K, R, dtype):
    print(f"case: {M}x{N}x{K} R={R} {dtype}", flush=True)
    x = synthetic.custom_inputs(M, N, K, R, seed=M + N + K + R, dtype=dtype, fmt="mxfp4")
    y, T = full_reference(x, "mxfp4")
    assert_parity(bits(run(x)), y, T, f"{M}x{N}x{K} R{R} {dtype}", dtype)


@pytest.mark.parametrize("M,N,K,R", [(1, 4112, 288, 5), (20, 4113, 2080, 33), (32, 8200, 416, 0), (33, 4100, 1056, 40),
                                     (64, 8193, 2208, 17), (50, 8300, 96, 8), (64, 4097, 3104, 0),
                                     (9, 1023, 608, 9), (30, 1025, 1056, 32), (3, 2817, 12288, 20), (17, 3841, 160, 1)])
def test_columns_of_a_workgroup(M, N, K, R):
    """Column counts around which a workgroup takes more or fewer columns, a wave more or fewer runs."""
    print(f"case: {M}x{N}x{K} R={R}", flush=True)
    x = synthetic.custom_inputs(M, N, K, R, seed=M + N + K + R, fmt="mxfp4")
    y, T = full_reference(x, "mxfp4")
    assert_parity(bits(run(x)), y, T, f"{M}x{N}x{K} R{R}", "bf16")


def test_nan_scales_and_zero_scales():
    x = synthetic.custom_inputs(5, 40, 416, 16, seed=11, fmt="mxfp4")
    x["ascales"][2, 3] = 255
    x["wscales"][12, 17] = 255
    x["wscales"][:, 20] = 0
    y, T = full_reference(x, "mxfp4")
    assert np.isnan(y[3]).all() and np.isnan(y[:, 17]).all()
    assert_parity(bits(run(x)), y, T, "NaN scales")


def test_agrees_with_gemm_mxfp4_and_repeats():
    x = synthetic.custom_inputs(24, 384, 1024, 32, seed=12, fmt="mxfp4")
    d = to_device(x)
    a = [d[k] for k in ARGS]
    few, again, many = w4.gemm_mxfp4_few(*a), w4.gemm_mxfp4_few(*a), w4.gemm_mxfp4(*a)
    assert torch.equal(few, again)
    y, T = full_reference(x, "mxfp4")
    assert_parity(bits(few), y, T, "few")
    assert_parity(bits(many), y, T, "many")


@pytest.mark.parametrize("shift", [1, 3, 8])
def test_unaligned_operands_and_guard(shift):
    """Scales, LoRA operands and out at odd addresses inside larger buffers: the
    result is the same and nothing around out changes."""
    x = synthetic.custom_inputs(19, 77, 288, 21, seed=13, fmt="mxfp4")
    d = to_device(x)
    want = w4.gemm_mxfp4_few(*(d[k] for k in ARGS))

    def moved(t):
        u = torch.zeros(t.numel() + 64, dtype=t.dtype, device=DEV)[shift:shift + t.numel()].view(t.shape)
        u.copy_(t)
        return u

    for k in ("ascales", "wscales", "lora_act_in", "lora_up", "wcscale", "bias"):
        d[k] = moved(d[k])
    buf = torch.full((19 * 77 + 128,), 7.0, dtype=torch.bfloat16, device=DEV)
    out = buf[64 + shift:64 + shift + 19 * 77].view(19, 77)
    w4.gemm_mxfp4_few(*(d[k] for k in ARGS), out=out)
    assert torch.equal(out, want)
    assert (buf[:64 + shift] == 7).all() and (buf[64 + shift + 19 * 77:] == 7).all()


def test_graph():
    x = synthetic.custom_inputs(8, 512, 1024, 16, seed=14, fmt="mxfp4")
    d = to_device(x)
    a = [d[k] for k in ARGS]
    la = d["lora_act_in"].clone()
    g = torch.cuda.CUDAGraph()
    a[6] = la
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        kept = w4.gemm_mxfp4_few(*a)
    for i in range(3):
        la.copy_(d["lora_act_in"] * (i + 1))
        g.replay()
        eager = w4.gemm_mxfp4_few(*a)
        torch.cuda.synchronize()
        assert torch.equal(kept, eager)
