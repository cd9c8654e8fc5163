"""A stream of another device than the tensors' is refused (CPU: tensors and streams
are stand-ins, and the native step is recorded)."""
from types import SimpleNamespace

import pytest
import torch

import bit_quantized_gemm_amd as w4

FIRST = {"quantize_mxfp4_act": 1, "gemm_mxfp4_few": 6, "rotary_axes": 4, "cross_attention": 3}


@pytest.fixture
def reached(monkeypatch):
    seen = []

    class Recorder:
        def __getattr__(self, fn):
            return lambda *args: seen.append(fn)

    class Current:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            seen.append(self.stream)

        def __exit__(self, *a):
            return False

    monkeypatch.setattr(w4._native, "binding", lambda: Recorder())
    monkeypatch.setattr(torch.cuda, "stream", Current)
    return seen


@pytest.mark.parametrize("name", FIRST)
def test_other_device(name, reached):
    tensor = SimpleNamespace(device=torch.device("cuda:0"))
    args = [tensor] * FIRST[name]
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        getattr(w4, name)(*args, stream=SimpleNamespace(cuda_stream=64, device=torch.device("cuda:1")))
    assert not reached
    here = SimpleNamespace(cuda_stream=64, device=torch.device("cuda:0"))
    getattr(w4, name)(*args, stream=here)
    assert reached == [here, name]
