"""A stream of another device than the tensors' is refused by the operators for many requests (CPU:
tensors and streams are stand-ins, and the native step is recorded)."""
from types import SimpleNamespace

import pytest
import torch

import bit_quantized_gemm_amd as w4

FIRST = {"block_norm": 1, "lora_adapters": 5, "cache_append": 5, "packed_attention": 4, "paged_attention": 5}


@pytest.mark.parametrize("name", FIRST)
def test_other_device(name, monkeypatch):
    seen = []

    class Recorder:
        def __getattr__(self, fn):
            return lambda *args: seen.append(fn)

    monkeypatch.setattr(w4._native, "binding", lambda: Recorder())
    args = [SimpleNamespace(device=torch.device("cuda:0"))] * FIRST[name]
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        getattr(w4, name)(*args, stream=SimpleNamespace(cuda_stream=0, device=torch.device("cuda:1")))
    assert not seen
    getattr(w4, name)(*args)
    assert seen == [name]
