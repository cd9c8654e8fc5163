"""The stream that the block operators work on (MI355X): torch's current one, a
torch stream, or a raw handle, of which 0 is the default stream."""
import pytest
import torch

import bit_quantized_gemm_amd as w4

DEV = "cuda:0"
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["quantize_mxfp4_act", "gemm_mxfp4_few", "rotary_axes", "cross_attention"])
def test_handle_that_the_native_step_sees(name, monkeypatch):
    seen = []

    class Recorder:
        def __getattr__(self, fn):
            return lambda *args: seen.append((fn, torch._C._cuda_getCurrentRawStream(0)))

    monkeypatch.setattr(w4._native, "binding", lambda: Recorder())
    some = {"quantize_mxfp4_act": 1, "gemm_mxfp4_few": 6, "rotary_axes": 4, "cross_attention": 3}[name]
    args = [torch.zeros(1, device=DEV)] * some
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = torch.cuda.Stream()
        for stream, want in ((None, side), (0, torch.cuda.default_stream()), (torch.cuda.default_stream(), torch.cuda.default_stream()),
                             (other, other), (other.cuda_stream, other)):
            getattr(w4, name)(*args, stream=stream)
            assert seen.pop() == (name, want.cuda_stream), stream


def test_default_stream_by_handle_keeps_order():
    """Work on the default stream by handle 0 comes after what was enqueued there before."""
    x = torch.zeros(1, 512, 8, 128, dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(512, 1, dtype=torch.int32, device=DEV)
    freq = torch.ones(64, device=DEV)
    big = torch.randn(4096, 4096, device=DEV)
    torch.cuda.synchronize()
    for i in range(5):
        for _ in range(4):
            big = (big @ big).clamp(-1, 1)                 # milliseconds of work ahead
        x.copy_((big[:512, :1024] * 0 + i).to(x.dtype).view(x.shape))
        y = w4.rotary_axes(x, pos, freq, (64,), stream=0)
        assert (y == i).all()
