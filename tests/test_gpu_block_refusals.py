"""What the block operators' Python entry points refuse when the tensors are on the
device (MI355X): every check of types, shapes, devices, strides and sizes raises before
anything is enqueued, and a call with none of the faults works."""
import pytest
import torch

import bit_quantized_gemm_amd as w4

DEV = "cuda:0"
BF, F16 = torch.bfloat16, torch.float16
pytestmark = pytest.mark.gpu


def zeros(*shape, dtype=BF, device=DEV):
    return torch.zeros(shape, dtype=dtype, device=device)


def byte(*shape):
    return zeros(*shape, dtype=torch.uint8)


def every_other(*shape, dtype=BF):
    """A tensor of this shape whose last dimension is not dense."""
    return zeros(*shape[:-1], 2 * shape[-1], dtype=dtype)[..., ::2]


def case(name, error, code=None, **over):
    return pytest.param(over, error, code, id=name)


def refused(fn, args, over, error, code):
    args = {**args, **{k: v() if callable(v) else v for k, v in over.items()}}
    with pytest.raises(error) as e:
        fn(**args)
    if code is not None:
        assert e.value.code == getattr(w4, code)


# ---------------------------------------------------------------- quantize_mxfp4_act

def quantize_args():
    return dict(x=zeros(4, 64), lora_down=zeros(8, 64))


@pytest.mark.parametrize("over,error,code", [
    case("x float32", TypeError, x=lambda: zeros(4, 64, dtype=torch.float32)),
    case("x not a tensor", TypeError, x=3),
    case("x on the host", ValueError, x=lambda: zeros(4, 64, device="cpu")),
    case("x 1-D", ValueError, x=lambda: zeros(64)),
    case("x strided", ValueError, x=lambda: every_other(4, 64)),
    case("x transposed", ValueError, x=lambda: zeros(64, 4).t()),
    case("lora_down of another type", TypeError, lora_down=lambda: zeros(8, 64, dtype=F16)),
    case("lora_down 1-D", ValueError, lora_down=lambda: zeros(64)),
    case("lora_down of another K", ValueError, lora_down=lambda: zeros(8, 32)),
    case("lora_down strided", ValueError, lora_down=lambda: every_other(8, 64)),
    case("lora_down on the host", ValueError, lora_down=lambda: zeros(8, 64, device="cpu")),
    case("act too small", ValueError, act=lambda: byte(4, 31)),
    case("act of rows too few", ValueError, act=lambda: byte(3, 32)),
    case("act strided", ValueError, act=lambda: every_other(4, 32, dtype=torch.uint8)),
    case("act of another type", TypeError, act=lambda: zeros(4, 32, dtype=torch.int8)),
    case("act on the host", ValueError, act=lambda: zeros(4, 32, dtype=torch.uint8, device="cpu")),
    case("ascales too small", ValueError, ascales=lambda: byte(1, 4)),
    case("ascales transposed", ValueError, ascales=lambda: byte(4, 2)),
    case("ascales of another type", TypeError, ascales=lambda: zeros(2, 4)),
    case("lora_act_in too small", ValueError, lora_act_in=lambda: zeros(4, 7)),
    case("lora_act_in of another type", TypeError, lora_act_in=lambda: zeros(4, 8, dtype=F16)),
    case("K past a block", w4.GemmError, "EINVAL", x=lambda: zeros(4, 48), lora_down=None),
    case("no rows", w4.GemmError, "EINVAL", x=lambda: zeros(0, 64)),
    case("too many ranks", w4.GemmError, "EINVAL", lora_down=lambda: zeros(129, 64))])
def test_quantize(over, error, code):
    refused(w4.quantize_mxfp4_act, quantize_args(), over, error, code)


def test_quantize_overlap():
    x = zeros(4, 64)
    with pytest.raises(w4.GemmError) as e:
        w4.quantize_mxfp4_act(x, act=x.view(-1).view(torch.uint8)[:128].view(4, 32))
    assert e.value.code == w4.EOVERLAP


# ---------------------------------------------------------------- gemm_mxfp4_few

def few_args():
    return dict(act=byte(4, 32), ascales=byte(2, 4), wgt=byte(16, 32), wscales=byte(2, 16),
                wcscale=zeros(16, dtype=torch.float32), bias=zeros(16, dtype=torch.float32),
                lora_act_in=zeros(4, 8), lora_up=zeros(8, 16))


FEW_SHAPES = dict(act=(4, 32), ascales=(2, 4), wgt=(16, 32), wscales=(2, 16), wcscale=(16,), bias=(16,),
                  lora_act_in=(4, 8), lora_up=(8, 16), out=(4, 16))


@pytest.mark.parametrize("name", FEW_SHAPES)
def test_few_operands(name):
    """Each operand smaller, larger, strided, of another type, on the host."""
    shape = FEW_SHAPES[name]
    dtype = torch.float32 if name in ("wcscale", "bias") else BF if name in ("lora_act_in", "lora_up", "out") else torch.uint8
    rows_follow = name in ("act", "wgt")       # whose shape the others are held to
    for d in (-1, 1):
        for i in range(len(shape)):
            wrong = tuple(n + d * (i == j) for j, n in enumerate(shape))
            refused(w4.gemm_mxfp4_few, few_args(), {name: zeros(*wrong, dtype=dtype)}, ValueError, None)
    refused(w4.gemm_mxfp4_few, few_args(), {name: every_other(*shape, dtype=dtype)}, ValueError, None)
    if len(shape) == 2 and not rows_follow:
        refused(w4.gemm_mxfp4_few, few_args(), {name: zeros(*shape[::-1], dtype=dtype)}, ValueError, None)
    refused(w4.gemm_mxfp4_few, few_args(), {name: zeros(*shape, dtype=torch.int64)}, TypeError, None)
    refused(w4.gemm_mxfp4_few, few_args(), {name: zeros(*shape, dtype=dtype, device="cpu")}, ValueError, None)


@pytest.mark.parametrize("over,error,code", [
    case("lora_act_in alone", ValueError, lora_up=None),
    case("lora_up alone", ValueError, lora_act_in=None),
    case("act 1-D", ValueError, act=lambda: byte(128)),
    case("lora_act_in 1-D", ValueError, lora_act_in=lambda: zeros(32)),
    case("dtype a text", TypeError, dtype="bf16"),
    case("dtype float32", TypeError, dtype=torch.float32),
    case("dtype not that of the LoRA term", TypeError, dtype=F16),
    case("out not of the dtype", TypeError, out=lambda: zeros(4, 16, dtype=F16), dtype=BF),
    case("wgt None", TypeError, wgt=None),
    case("K past a block", w4.GemmError, "EINVAL", act=lambda: byte(4, 24), wgt=lambda: byte(16, 24),
         ascales=lambda: byte(1, 4), wscales=lambda: byte(1, 16)),
    case("65 rows", w4.GemmError, "EINVAL", act=lambda: byte(65, 32), ascales=lambda: byte(2, 65), lora_act_in=lambda: zeros(65, 8)),
    case("no rows", w4.GemmError, "EINVAL", act=lambda: byte(0, 32), ascales=lambda: byte(2, 0), lora_act_in=lambda: zeros(0, 8))])
def test_few(over, error, code):
    refused(w4.gemm_mxfp4_few, few_args(), over, error, code)


# ---------------------------------------------------------------- rotary_axes

def rotary_args():
    return dict(x=zeros(2, 3, 4, 16), positions=zeros(2, 3, 2, dtype=torch.int32),
                inv_freq=zeros(8, dtype=torch.float32), sections=(5, 3))


@pytest.mark.parametrize("over,error,code", [
    case("x float32", TypeError, x=lambda: zeros(2, 3, 4, 16, dtype=torch.float32)),
    case("x on the host", ValueError, x=lambda: zeros(2, 3, 4, 16, device="cpu")),
    case("x 3-D", ValueError, x=lambda: zeros(2, 3, 64)),
    case("x last dimension strided", ValueError, x=lambda: every_other(2, 3, 4, 16)),
    case("positions int64", TypeError, positions=lambda: zeros(2, 3, 2, dtype=torch.int64)),
    case("positions too few tokens", ValueError, positions=lambda: zeros(2, 2, 2, dtype=torch.int32)),
    case("positions too few batches", ValueError, positions=lambda: zeros(1, 3, 2, dtype=torch.int32)),
    case("positions too few axes", ValueError, positions=lambda: zeros(2, 3, 1, dtype=torch.int32)),
    case("positions last dimension strided", ValueError, positions=lambda: every_other(2, 3, 2, dtype=torch.int32)),
    case("positions on the host", ValueError, positions=lambda: zeros(2, 3, 2, dtype=torch.int32, device="cpu")),
    case("inv_freq float64", TypeError, inv_freq=lambda: zeros(8, dtype=torch.float64)),
    case("inv_freq too short", ValueError, inv_freq=lambda: zeros(7, dtype=torch.float32)),
    case("inv_freq too long", ValueError, inv_freq=lambda: zeros(9, dtype=torch.float32)),
    case("inv_freq strided", ValueError, inv_freq=lambda: every_other(8, dtype=torch.float32)),
    case("inv_freq on the host", ValueError, inv_freq=lambda: zeros(8, dtype=torch.float32, device="cpu")),
    case("sections a number", TypeError, sections=8),
    case("no axes", ValueError, sections=()),
    case("five axes", ValueError, sections=(1, 1, 1, 1, 4), positions=lambda: zeros(2, 3, 5, dtype=torch.int32)),
    case("a section below 0 at the end", ValueError, sections=(8, -1)),
    case("more pairs than a head has", w4.GemmError, "EINVAL", sections=(6, 3), inv_freq=lambda: zeros(9, dtype=torch.float32)),
    case("head too large", w4.GemmError, "EINVAL", x=lambda: zeros(2, 3, 4, 258)),
    case("odd head, interleaved", w4.GemmError, "EINVAL", x=lambda: zeros(2, 3, 4, 17)),
    case("odd address, interleaved", w4.GemmError, "EALIGN", x=lambda: zeros(385)[1:].view(2, 3, 4, 16)),
    case("out of another type", TypeError, out=lambda: zeros(2, 3, 4, 16, dtype=F16)),
    case("out too small", ValueError, out=lambda: zeros(2, 3, 3, 16)),
    case("out last dimension strided", ValueError, out=lambda: every_other(2, 3, 4, 16)),
    case("out on the host", ValueError, out=lambda: zeros(2, 3, 4, 16, device="cpu")),
    case("out repeats memory", w4.GemmError, "EINVAL", out=lambda: zeros(1, 3, 4, 16).expand(2, 3, 4, 16))])
def test_rotary(over, error, code):
    refused(w4.rotary_axes, rotary_args(), over, error, code)


def test_rotary_overlap():
    buf = zeros(1000)
    x, moved = buf[:384].view(2, 3, 4, 16), buf[8:392].view(2, 3, 4, 16)
    with pytest.raises(w4.GemmError) as e:
        w4.rotary_axes(**{**rotary_args(), "x": x}, out=moved)
    assert e.value.code == w4.EOVERLAP


# ---------------------------------------------------------------- cross_attention

def attention_args():
    return dict(q=zeros(2, 3, 4, 64), k=zeros(2, 5, 2, 64), v=zeros(2, 5, 2, 64))


@pytest.mark.parametrize("over,error,code", [
    case("q float32", TypeError, q=lambda: zeros(2, 3, 4, 64, dtype=torch.float32)),
    case("q on the host", ValueError, q=lambda: zeros(2, 3, 4, 64, device="cpu")),
    case("q 3-D", ValueError, q=lambda: zeros(2, 3, 256)),
    case("q last dimension strided", ValueError, q=lambda: every_other(2, 3, 4, 64)),
    case("k 3-D", ValueError, k=lambda: zeros(2, 5, 128)),
    case("k of another type", TypeError, k=lambda: zeros(2, 5, 2, 64, dtype=F16)),
    case("k of another batch", ValueError, k=lambda: zeros(1, 5, 2, 64)),
    case("k of another head size", ValueError, k=lambda: zeros(2, 5, 2, 56)),
    case("k on the host", ValueError, k=lambda: zeros(2, 5, 2, 64, device="cpu")),
    case("k last dimension strided", ValueError, k=lambda: every_other(2, 5, 2, 64)),
    case("v shorter than k", ValueError, v=lambda: zeros(2, 4, 2, 64)),
    case("v of other heads", ValueError, v=lambda: zeros(2, 5, 1, 64)),
    case("v of another type", TypeError, v=lambda: zeros(2, 5, 2, 64, dtype=F16)),
    case("v on the host", ValueError, v=lambda: zeros(2, 5, 2, 64, device="cpu")),
    case("kv_lens int64", TypeError, kv_lens=lambda: zeros(2, dtype=torch.int64)),
    case("kv_lens too short", ValueError, kv_lens=lambda: zeros(1, dtype=torch.int32)),
    case("kv_lens 2-D", ValueError, kv_lens=lambda: zeros(2, 1, dtype=torch.int32)),
    case("kv_lens strided", ValueError, kv_lens=lambda: every_other(2, dtype=torch.int32)),
    case("kv_lens on the host", ValueError, kv_lens=lambda: zeros(2, dtype=torch.int32, device="cpu")),
    case("kv_lens a list", TypeError, kv_lens=[5, 5]),
    case("scale a text", TypeError, scale="0.1"),
    case("scale 0", w4.GemmError, "EINVAL", scale=0.0),
    case("scale below 0", w4.GemmError, "EINVAL", scale=-0.125),
    case("scale NaN", w4.GemmError, "EINVAL", scale=float("nan")),
    case("scale infinite", w4.GemmError, "EINVAL", scale=float("inf")),
    case("heads that do not divide", w4.GemmError, "EINVAL", q=lambda: zeros(2, 3, 5, 64)),
    case("head size 20", w4.GemmError, "EINVAL", q=lambda: zeros(2, 3, 4, 20), k=lambda: zeros(2, 5, 2, 20), v=lambda: zeros(2, 5, 2, 20)),
    case("head size 136", w4.GemmError, "EINVAL", q=lambda: zeros(2, 3, 4, 136), k=lambda: zeros(2, 5, 2, 136), v=lambda: zeros(2, 5, 2, 136)),
    case("token stride not a multiple of 8", w4.GemmError, "EINVAL", k=lambda: zeros(2, 5, 132)[..., :128].unflatten(-1, (2, 64))),
    case("address not on 16 bytes", w4.GemmError, "EALIGN", v=lambda: zeros(1284)[4:].view(2, 5, 2, 64)),
    case("out of another type", TypeError, out=lambda: zeros(2, 3, 4, 64, dtype=F16)),
    case("out too small", ValueError, out=lambda: zeros(2, 2, 4, 64)),
    case("out on the host", ValueError, out=lambda: zeros(2, 3, 4, 64, device="cpu")),
    case("out last dimension strided", ValueError, out=lambda: every_other(2, 3, 4, 64)),
    case("out repeats memory", w4.GemmError, "EINVAL", out=lambda: zeros(1, 3, 4, 64).expand(2, 3, 4, 64))])
def test_attention(over, error, code):
    refused(w4.cross_attention, attention_args(), over, error, code)


def test_attention_overlap():
    q = zeros(2, 3, 4, 64)
    with pytest.raises(w4.GemmError) as e:
        w4.cross_attention(q, q[:, :, :2], q[:, :, 2:], out=q)
    assert e.value.code == w4.EOVERLAP


def test_calls_without_a_fault():
    assert w4.quantize_mxfp4_act(**quantize_args())[2].shape == (4, 8)
    assert w4.gemm_mxfp4_few(**few_args()).shape == (4, 16)
    assert w4.rotary_axes(**rotary_args()).shape == (2, 3, 4, 16)
    assert w4.cross_attention(**attention_args()).shape == (2, 3, 4, 64)
