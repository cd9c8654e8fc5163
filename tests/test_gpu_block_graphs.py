"""rotary_axes and gemm_mxfp4_few on a stream of the caller's and replayed from a graph
(MI355X): every replay gives what the eager call gives for the inputs of that moment."""
import pytest
import torch

import bit_quantized_gemm_amd as w4
import synthetic

from gpu_helpers import ARGS, to_device

DEV = "cuda:0"
pytestmark = pytest.mark.gpu


def rotary_inputs(interleaved):
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(2, 300, 9, 72, generator=g, device=DEV).bfloat16()
    pos = torch.randint(0, 64, (2, 300, 3), generator=g, device=DEV, dtype=torch.int32)
    freq = torch.rand(32, generator=g, device=DEV)
    return x, pos, freq, dict(sections=(4, 11, 17), interleaved=interleaved)


@pytest.mark.parametrize("interleaved", [True, False])
def test_rotary_on_another_stream(interleaved):
    x, pos, freq, kw = rotary_inputs(interleaved)
    want = w4.rotary_axes(x, pos, freq, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        here = x.clone()
    for stream in (side, side.cuda_stream):
        got = w4.rotary_axes(x, pos, freq, stream=stream, **kw)
        side.synchronize()
        assert torch.equal(got, want)
    w4.rotary_axes(here, pos, freq, out=here, stream=side, **kw)      # after the copy, in its stream
    side.synchronize()
    assert torch.equal(here, want)


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("in_place", [True, False])
def test_rotary_in_a_graph(in_place, interleaved):
    x, pos, freq, kw = rotary_inputs(interleaved)
    sx, sp = x.clone(), pos.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = w4.rotary_axes(sx, sp, freq, out=sx if in_place else None, **kw)
    for i in range(4):
        sx.copy_(x * (i + 1))
        sp.copy_(pos + 7 * i)
        g.replay()
        eager = w4.rotary_axes(x * (i + 1), pos + 7 * i, freq, **kw)
        torch.cuda.synchronize()
        assert torch.equal(kept, eager) and (not in_place or kept.data_ptr() == sx.data_ptr())


@pytest.mark.parametrize("M,N", [(1, 512), (24, 4200), (64, 300)])
def test_few_rows_on_another_stream(M, N):
    d = to_device(synthetic.custom_inputs(M, N, 1056, 20, seed=M + N, fmt="mxfp4"))
    a = [d[k] for k in ARGS]
    want = w4.gemm_mxfp4_few(*a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        got = w4.gemm_mxfp4_few(*a, stream=stream)
        side.synchronize()
        assert torch.equal(got, want)
    with torch.cuda.stream(side):                # inputs made on the stream just before the call
        moved = [t.clone() for t in a]
        got = w4.gemm_mxfp4_few(*moved)
    side.synchronize()
    assert torch.equal(got, want)
