"""What quantize_mxfp4_act, gemm_mxfp4_few, rotary_axes and cross_attention refuse,
before anything is enqueued (CPU: no call here reaches a launch), and their
workspace rules."""
import ctypes

import pytest
import torch

import bit_quantized_gemm_amd as w4

REACHED = (w4.OK, w4.EDEVICE, w4.ELAUNCH)   # checks passed; only the device check is left here


# ---------------------------------------------------------------- quantize_mxfp4_act

def quant(f16=False, **over):
    a = dict(x=0x10000, lora_down=0x2000000, act=0x3000000, ascales=0x4000000, lora_act_in=0x5000000,
             M=64, K=128, R=16, workspace=0, workspace_bytes=0)
    a.update(over)
    return w4.quantize_mxfp4_raw(f16, *a.values(), 0)


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("over,code", [
    (dict(M=0), "EINVAL"), (dict(K=0), "EINVAL"), (dict(K=16), "EINVAL"), (dict(K=48), "EINVAL"), (dict(R=-1), "EINVAL"),
    (dict(R=129), "EINVAL"), (dict(M=1 << 20, K=1 << 11), "EINVAL"), (dict(x=0), "EINVAL"), (dict(act=0), "EINVAL"),
    (dict(ascales=0), "EINVAL"), (dict(lora_down=0), "EINVAL"), (dict(lora_act_in=0), "EINVAL"),
    (dict(x=0x10008), "EALIGN"), (dict(lora_down=0x2000002), "EALIGN"), (dict(act=0x3000008), "EALIGN"),
    (dict(lora_act_in=0x5000001), "EALIGN"), (dict(act=0x10010), "EOVERLAP"), (dict(ascales=0x3000001), "EOVERLAP"),
    (dict(lora_act_in=0x2000010), "EOVERLAP"), (dict(K=12288, M=16), "ESCRATCH"),
    (dict(K=12288, M=16, workspace=0x6000000, workspace_bytes=64), "ESCRATCH"),
    (dict(K=12288, M=16, workspace=0x6000008, workspace_bytes=1 << 24), "EALIGN"),
    (dict(K=12288, M=16, workspace=0x10000, workspace_bytes=1 << 24), "EOVERLAP")])
def test_quantize_refuses(over, code, f16):
    assert quant(f16, **over) == getattr(w4, code)


def test_quantize_accepts():
    assert quant(R=0, lora_down=0, lora_act_in=0) in REACHED
    assert quant(K=12288, M=16, workspace=0x6000000, workspace_bytes=1 << 24) in REACHED


def test_quantize_workspace():
    assert w4.quantize_mxfp4_workspace(4096, 3072, 16) == 0          # rows fill the chip
    assert w4.quantize_mxfp4_workspace(16, 12288, 0) == 0            # no sums to join
    assert w4.quantize_mxfp4_workspace(16, 12288, 32) > 0
    for bad in ((0, 32, 0), (1, 48, 0), (1, 32, 129)):
        with pytest.raises(ValueError):
            w4.quantize_mxfp4_workspace(*bad)


# ---------------------------------------------------------------- gemm_mxfp4_few

def few(f16=False, **over):
    a = dict(act=0x10000, ascales=0x20000, wgt=0x30000, wscales=0x40000, wcscale=0x50000, bias=0x60000,
             lora_act_in=0x70000, lora_up=0x80000, out=0x90000000, M=16, N=64, K=128, R=16)
    a.update(over)
    return w4.gemm_mxfp4_few_raw(f16, *a.values(), 0)


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("over,code", [
    (dict(M=0), "EINVAL"), (dict(M=65), "EINVAL"), (dict(N=0), "EINVAL"), (dict(K=16), "EINVAL"), (dict(K=80), "EINVAL"),
    (dict(R=-1), "EINVAL"), (dict(R=1025), "EINVAL"), (dict(N=1 << 20, K=1 << 12), "EINVAL"), (dict(act=0), "EINVAL"),
    (dict(wscales=0), "EINVAL"), (dict(lora_up=0), "EINVAL"), (dict(act=0x10008), "EALIGN"), (dict(wgt=0x30004), "EALIGN"),
    (dict(bias=0x60002), "EALIGN"), (dict(out=0x90000001), "EALIGN"), (dict(wgt=0x90000010), "EOVERLAP"),
    (dict(lora_up=0x90000010), "EOVERLAP")])
def test_few_refuses(over, code, f16):
    assert few(f16, **over) == getattr(w4, code)


def test_few_accepts():
    assert few(M=64, R=0, lora_act_in=0, lora_up=0) in REACHED


# ---------------------------------------------------------------- rotary_axes

def rot(**over):
    a = dict(x=0x10000000, out=0x20000000, positions=0x30000000, inv_freq=0x40000000, batch=2, tokens=4, heads=3,
             head_dim=16, axes=2, sections=(4, 4, 0, 0), x_stride=(192, 48, 16), out_stride=(192, 48, 16),
             pos_stride=(8, 2), interleaved=1, inverse=0, f16=0)
    a.update(over)
    return w4.rotary_axes_raw(w4.RotaryArgs(*a.values()), 0)


@pytest.mark.parametrize("over,code", [
    (dict(batch=-1), "EINVAL"), (dict(tokens=-1), "EINVAL"), (dict(heads=-1), "EINVAL"), (dict(head_dim=0), "EINVAL"),
    (dict(head_dim=257), "EINVAL"), (dict(axes=0), "EINVAL"), (dict(axes=5), "EINVAL"), (dict(sections=(4, 5, 0, 0)), "EINVAL"),
    (dict(sections=(-1, 4, 0, 0)), "EINVAL"), (dict(sections=(2**31 - 1, 2, 0, 0)), "EINVAL"), (dict(f16=2), "EINVAL"),
    (dict(interleaved=2), "EINVAL"), (dict(head_dim=15, sections=(3, 4, 0, 0)), "EINVAL"), (dict(batch=70000), "EINVAL"),
    (dict(x_stride=(192, 48, -16)), "EINVAL"), (dict(x_stride=(2**62, 48, 16)), "EINVAL"),
    (dict(out_stride=(192, 48, 0)), "EINVAL"), (dict(out_stride=(192, 48, 8)), "EINVAL"), (dict(out_stride=(0, 48, 16)), "EINVAL"),
    (dict(x=0), "EINVAL"), (dict(out=0), "EINVAL"), (dict(positions=0), "EINVAL"), (dict(inv_freq=0), "EINVAL"),
    (dict(x=0x10000001), "EALIGN"), (dict(out=0x20000002), "EALIGN"), (dict(positions=0x30000002), "EALIGN"),
    (dict(inv_freq=0x40000001), "EALIGN"), (dict(x_stride=(192, 49, 16)), "EALIGN"), (dict(out=0x10000020), "EOVERLAP"),
    (dict(out=0x10000000, out_stride=(384, 96, 16)), "EOVERLAP"), (dict(positions=0x20000010), "EOVERLAP"),
    (dict(inv_freq=0x20000010), "EOVERLAP")])
def test_rotary_refuses(over, code):
    assert rot(**over) == getattr(w4, code)


@pytest.mark.parametrize("over", [
    dict(), dict(out=0x10000000), dict(x_stride=(0, 0, 0)), dict(interleaved=0, x=0x10000002), dict(pos_stride=(0, 2)),
    dict(batch=1, out_stride=(0, 48, 16)), dict(sections=(0, 0, 0, 0), inv_freq=0), dict(x_stride=(16, 32, 128))])
def test_rotary_accepts(over):
    assert rot(**over) in REACHED


def test_rotary_empty_is_ok():
    assert rot(tokens=0, x=0, out=0) == w4.OK and rot(heads=0) == w4.OK and rot(batch=0) == w4.OK
    assert w4.rotary_axes_raw(w4.RotaryArgs(), 0) == w4.EINVAL


# ---------------------------------------------------------------- cross_attention

def attn(**over):
    a = dict(q=0x10000000, k=0x20000000, v=0x30000000, out=0x40000000, lse=0, kv_lens=0, batch=2, q_len=200, kv_len=6,
             q_heads=4, kv_heads=2, head_dim=64, q_stride=(51200, 256, 64), k_stride=(768, 128, 64),
             v_stride=(768, 128, 64), out_stride=(51200, 256, 64), scale=0.125, f16=0, workspace=0, workspace_bytes=0)
    a.update(over)
    return w4.AttentionArgs(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(batch=-1), "EINVAL"), (dict(q_len=-1), "EINVAL"), (dict(kv_len=-1), "EINVAL"), (dict(q_heads=-2), "EINVAL"),
    (dict(kv_heads=0), "EINVAL"), (dict(q_heads=5), "EINVAL"), (dict(head_dim=0), "EINVAL"), (dict(head_dim=20), "EINVAL"),
    (dict(head_dim=136), "EINVAL"), (dict(scale=0.0), "EINVAL"), (dict(scale=-1.0), "EINVAL"),
    (dict(scale=float("nan")), "EINVAL"), (dict(scale=float("inf")), "EINVAL"), (dict(f16=2), "EINVAL"),
    (dict(q_stride=(51200, 256, 68)), "EINVAL"), (dict(k_stride=(768, -128, 64)), "EINVAL"),
    (dict(k_stride=(768, 1 << 23, 64)), "EINVAL"), (dict(v_stride=(770, 128, 64)), "EINVAL"),
    (dict(out_stride=(51200, 256, 0)), "EINVAL"), (dict(out_stride=(51200, 64, 64)), "EINVAL"),
    (dict(q=0), "EINVAL"), (dict(k=0), "EINVAL"), (dict(v=0), "EINVAL"), (dict(out=0), "EINVAL"),
    (dict(q=0x10000008), "EALIGN"), (dict(k=0x20000002), "EALIGN"), (dict(out=0x40000004), "EALIGN"),
    (dict(lse=0x50000002), "EALIGN"), (dict(kv_lens=0x50000001), "EALIGN"), (dict(out=0x10000010), "EOVERLAP"),
    (dict(out=0x20000010), "EOVERLAP"), (dict(lse=0x40000100), "EOVERLAP"), (dict(kv_lens=0x40000100), "EOVERLAP"),
    (dict(lse=0x30000000), "EOVERLAP"), (dict(q_len=1 << 30), "EINVAL"), (dict(batch=1 << 24), "EINVAL"),
    (dict(q_len=1, kv_len=6000), "ESCRATCH"),
    (dict(q_len=1, kv_len=6000, workspace=0x60000000, workspace_bytes=8), "ESCRATCH"),
    (dict(q_len=1, kv_len=6000, workspace=0x60000008, workspace_bytes=1 << 24), "EALIGN"),
    (dict(q_len=1, kv_len=6000, workspace=0x20000000, workspace_bytes=1 << 24), "EOVERLAP")])
def test_attention_refuses(over, code):
    assert w4.cross_attention_raw(attn(**over), 0) == getattr(w4, code)


@pytest.mark.parametrize("over", [
    dict(), dict(kv_len=0, k=0, v=0), dict(k_stride=(0, 0, 0), v_stride=(0, 0, 0)), dict(lse=0x50000000, kv_lens=0x58000000),
    dict(batch=1, q_stride=(3, 256, 64)), dict(k=0x30000000), dict(kv_len=1, k_stride=(128, 5, 64)),
    dict(q_len=1, kv_len=6000, workspace=0x60000000, workspace_bytes=1 << 24)])
def test_attention_accepts(over):
    assert w4.cross_attention_raw(attn(**over), 0) in REACHED


def test_attention_empty_and_null():
    assert w4.cross_attention_raw(attn(batch=0, q=0), 0) == w4.OK
    assert w4.cross_attention_raw(attn(q_len=0), 0) == w4.OK and w4.cross_attention_raw(attn(q_heads=0), 0) == w4.OK
    lib = w4._native.load()
    assert lib.cross_attention(None, None) == w4.EINVAL and lib.rotary_axes(None, None) == w4.EINVAL
    assert lib.cross_attention_workspace(None) == w4.EINVAL


def test_attention_workspace():
    need = w4.cross_attention_workspace
    assert need(attn(q_len=1, kv_len=0)) == 0 and need(attn(batch=64, q_len=4096, kv_len=4096)) == 0
    assert need(attn(q_len=1, kv_len=100000)) > 0 and need(attn(head_dim=20)) == w4.EINVAL


# ---------------------------------------------------------------- the Python checks

def test_python_checks():
    bf, z = torch.bfloat16, torch.zeros
    with pytest.raises(TypeError):
        w4.quantize_mxfp4_act(z(4, 32))
    with pytest.raises(ValueError):
        w4.quantize_mxfp4_act(z(4, 32, dtype=bf))                      # not on a GPU
    with pytest.raises(TypeError):
        w4.rotary_axes(z(1, 1, 1, 8), z(1, 1, 1, dtype=torch.int32), z(2), (2,))
    with pytest.raises(ValueError):
        w4.cross_attention(*(z(1, 1, 1, 8, dtype=bf) for _ in range(3)))
    with pytest.raises(ValueError):
        w4.gemm_mxfp4_few(*(z(1, 16, dtype=torch.uint8) for _ in range(4)), z(1), z(1))


def test_structures_match_the_header(tmp_path):
    """Field offsets of the ctypes structures equal those a C compiler gives the header's."""
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    names = {"rotary_axes_t": w4.RotaryArgs, "cross_attention_t": w4.AttentionArgs}
    body = "".join(f'printf("%zu\\n", sizeof({t}));' + "".join(f'printf("%zu\\n", offsetof({t}, {f[0]}));' for f in c._fields_)
                   for t, c in names.items())
    src = tmp_path / "t.c"
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"gemm_w4a4.h\"\nint main(void) {" + body + "return 0;}")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", f"-I{root}/include", str(src), "-o", str(tmp_path / "t")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "t")], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for c in names.values():
        want += [ctypes.sizeof(c)] + [getattr(c, f[0]).offset for f in c._fields_]
    assert got == want

