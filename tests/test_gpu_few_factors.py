"""Column factors of gemm_mxfp4_few that a wave's part of a sum must not be multiplied by
(MI355X): infinite, NaN, and near float32's largest. The oracle's results within the
bound of gemm_mxfp4's tests, infinities with its sign, NaN where it has them."""
import numpy as np
import pytest
import torch

import bit_quantized_gemm_amd as w4
import synthetic

from gpu_helpers import ARGS, assert_parity, full_reference, to_device

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K,R", [(1, 40, 128, 0), (1, 40, 4096, 16), (8, 64, 4096, 300), (16, 1001, 32, 3), (20, 50, 2080, 128),
                                     (32, 4113, 1056, 17), (30, 8200, 416, 33), (64, 100, 3104, 40), (50, 4100, 1056, 0), (64, 8193, 544, 9)])
def test_factors(M, N, K, R, dtype):
    print(f"case: {M}x{N}x{K} R={R} {dtype}", flush=True)
    x = synthetic.custom_inputs(M, N, K, R, seed=M + N + K + R, dtype=dtype, fmt="mxfp4")
    wc = x["wcscale"]
    wc[3], wc[17], wc[20], wc[21], wc[22] = np.inf, -np.inf, np.nan, 2.0 ** 70, -2.0 ** 100
    wc[-1] = np.inf
    with np.errstate(invalid="ignore", over="ignore"):
        y, T = full_reference(x, "mxfp4")
    assert np.isinf(y[:, [3, 17, -1]]).all() and np.isnan(y[:, 20]).all()
    d = to_device(x)
    got = w4.gemm_mxfp4_few(*(d[k] for k in ARGS), dtype=torch.float16 if dtype == "f16" else torch.bfloat16)
    bits = got.view(torch.int16).cpu().numpy().view(np.uint16)
    with np.errstate(invalid="ignore", over="ignore"):
        assert_parity(bits, y, T, f"{M}x{N}x{K} R{R} {dtype}", dtype)


def test_infinite_lora_beside_an_infinite_factor():
    """inf from the factor and -inf from the LoRA term is NaN; apart, each is itself."""
    x = synthetic.custom_inputs(4, 32, 256, 2, seed=5, fmt="mxfp4")
    x["wcscale"][5] = np.inf
    x["lora_act_in"][:] = 0
    x["lora_act_in"][1, 0] = 0xFF80                    # -inf
    x["lora_up"][:] = 0x3F80                           # 1.0
    with np.errstate(invalid="ignore"):
        y, _ = full_reference(x, "mxfp4")
    d = to_device(x)
    got = w4.gemm_mxfp4_few(*(d[k] for k in ARGS)).double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(y)) and np.isinf(y[0, 5])
    assert np.array_equal(got[np.isinf(y)], y[np.isinf(y)])
