"""Sizes near 2^31 that cross_attention refuses, since rows and keys are counted in int
and rounded up to tiles (CPU: workspace sizes and refusals only)."""
import pytest

import bit_quantized_gemm_amd as w4

PAST_END = 1024


def args(**over):
    a = dict(q=0x10000000, k=0x20000000, v=0x30000000, out=1 << 40, lse=0, kv_lens=0, batch=1, q_len=1, kv_len=600,
             q_heads=1, kv_heads=1, head_dim=8, q_stride=(0, 0, 0), k_stride=(0, 0, 0), v_stride=(0, 0, 0),
             out_stride=(0, 8, 8), scale=0.125, f16=0, workspace=0, workspace_bytes=0)
    a.update(over)
    return w4.AttentionArgs(*a.values())


@pytest.mark.parametrize("over", [
    dict(q_len=2**31 - 1), dict(q_len=2**31 - 100), dict(q_len=2**31 - PAST_END + 1), dict(q_len=2**30 - 200, q_heads=2),
    dict(q_len=2**30 - 200, q_heads=2, kv_heads=2), dict(kv_len=2**31 - 1), dict(kv_len=2**31 - PAST_END + 1)], ids=str)
def test_refused(over):
    a = args(**over)
    assert w4.cross_attention_workspace(a) == w4.EINVAL
    assert w4.cross_attention_raw(a, 0) == w4.EINVAL


@pytest.mark.parametrize("over", [dict(q_len=2**31 - PAST_END), dict(kv_len=2**31 - PAST_END), dict(q_len=2**30 - 512, q_heads=2)], ids=str)
def test_largest(over):
    assert w4.cross_attention_workspace(args(**over)) >= 0
