"""What autograd sees of the block operators (MI355X): results are detached, and a
tensor given as an output has changed in place."""
import pytest
import torch

import bit_quantized_gemm_amd as w4

DEV = "cuda:0"
pytestmark = pytest.mark.gpu


def half(*shape, grad=False):
    return torch.randn(shape, device=DEV).bfloat16().requires_grad_(grad)


def byte(*shape):
    return torch.zeros(shape, dtype=torch.uint8, device=DEV)


def calls():
    """name -> (call with outputs given, the outputs, call without)"""
    x, down = half(4, 64, grad=True), half(8, 64, grad=True)
    act, asc, low = byte(4, 32), byte(2, 4), half(4, 8)
    codes = [t.fill_(0x21) for t in (byte(4, 32), byte(2, 4), byte(16, 32), byte(2, 16))]
    ones, up, y = torch.ones(16, device=DEV, requires_grad=True), half(8, 16, grad=True), half(4, 16)
    h, turned = half(1, 3, 2, 16, grad=True), half(1, 3, 2, 16)
    pos, freq = torch.zeros(3, 1, dtype=torch.int32, device=DEV), torch.ones(8, device=DEV)
    k, o = half(1, 5, 2, 16, grad=True), half(1, 3, 2, 16)
    return {"quantize_mxfp4_act": (lambda: w4.quantize_mxfp4_act(x, down, act, asc, low), (act, asc, low),
                                   lambda: w4.quantize_mxfp4_act(x, down)),
            "gemm_mxfp4_few": (lambda: w4.gemm_mxfp4_few(*codes, ones, ones, low, up, out=y), (y,),
                               lambda: w4.gemm_mxfp4_few(*codes, ones, ones, low, up)),
            "rotary_axes": (lambda: w4.rotary_axes(h, pos, freq, (8,), out=turned), (turned,),
                            lambda: w4.rotary_axes(h, pos, freq, (8,))),
            "cross_attention": (lambda: w4.cross_attention(h, k, k, out=o), (o,), lambda: w4.cross_attention(h, k, k))}


NAMES = ["quantize_mxfp4_act", "gemm_mxfp4_few", "rotary_axes", "cross_attention"]


@pytest.mark.parametrize("name", NAMES)
def test_given_outputs_move_on(name):
    given, outs, _ = calls()[name]
    was = [t._version for t in outs]
    given()
    assert [t._version for t in outs] == [v + 1 for v in was]
    assert not any(t.requires_grad for t in outs)


@pytest.mark.parametrize("name", NAMES)
def test_results_are_detached(name):
    r = calls()[name][2]()
    assert not any(t.requires_grad for t in (r if isinstance(r, tuple) else (r,)))


def test_backward_past_a_rotation_in_place_raises():
    """A value saved for the backward pass and then rotated where it is: an error, not a wrong gradient."""
    w = torch.ones(1, 3, 2, 16, device=DEV, dtype=torch.bfloat16, requires_grad=True)
    x = half(1, 3, 2, 16)
    loss = (w * x).sum()                          # saves x
    w4.rotary_axes(x, torch.ones(3, 1, dtype=torch.int32, device=DEV), torch.ones(8, device=DEV), (8,), out=x)
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()


def test_a_refused_call_changes_nothing():
    x = half(1, 3, 2, 16)
    was, before = x._version, x.clone()
    with pytest.raises(w4.GemmError):
        w4.rotary_axes(x, torch.ones(3, 1, dtype=torch.int32, device=DEV), torch.ones(9, device=DEV), (9,), out=x)   # 9 pairs of 16
    assert x._version == was and torch.equal(x, before)


def test_inference_tensors_as_outputs():
    with torch.inference_mode():
        x, out = half(1, 3, 2, 16), half(1, 3, 2, 16)
    pos, freq = torch.zeros(3, 1, dtype=torch.int32, device=DEV), torch.ones(8, device=DEV)
    for mode in (torch.inference_mode, torch.no_grad):
        with mode():
            assert torch.equal(w4.rotary_axes(x, pos, freq, (8,), out=out), x)
