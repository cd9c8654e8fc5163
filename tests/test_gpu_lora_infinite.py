"""lora_adapters where a row's sum over K is infinite for some rank (MI355X): its other sums, past
binary16's range too, keep their size, so that the result is the definition's signed infinity."""
import numpy as np
import pytest
import torch

import bit_quantized_gemm_amd as w4
import oracle.request_ref as ref

from block_helpers import DEV, TORCH, assert_within, values_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N", [(5, 72), (90, 1001), (2100, 2056)])     # few rows, and rows grouped by adapter
def test_infinite_beside_large(M, N, dtype):
    A, K, R = 3, 64, 12
    g = torch.Generator().manual_seed(M + N)
    x = torch.randn(M, K, generator=g)
    x[:, 0], x[:, 1] = 1.0, 1000.0
    down = torch.randn(A, R, K, generator=g) * 0.1
    down[:, 1, 1] = 1000.0                              # a sum of 1e6
    down[0, 0, 0] = float("inf")                        # adapter 0: one infinite sum
    down[1, 0, 0], down[1, 5, 0] = float("-inf"), float("inf")   # adapter 1: two, which meet in some columns
    up = torch.where(torch.rand(A, R, N, generator=g) < 0.5, -1.0, 1.0)
    y = torch.randn(M, N, generator=g)
    y, x, down, up = (t.to(TORCH[dtype]).to(DEV) for t in (y, x, down, up))
    ids = torch.from_numpy((np.arange(M) * 7 % 4 - 1).astype(np.int32)).to(DEV)
    got = values_of(w4.lora_adapters(y, x, down, up, ids))
    with np.errstate(invalid="ignore"):
        want, bound = ref.lora_adapters_ref(*(values_of(t) for t in (y, x, down, up)), ids.cpu().numpy(), dtype=dtype)
    assert np.isinf(want[ids.cpu().numpy() == 0]).all()
    if dtype == "f16":      # adapter 2's finite results of about 1e6: from 65504 + 16, half a spacing, on binary16 has an infinity
        want = np.where(np.abs(want) >= 65520, np.copysign(np.inf, want), want)
    assert_within(got, want, bound, f"{M}x{N} {dtype}")
