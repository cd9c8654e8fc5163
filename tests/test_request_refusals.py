"""What the operators for many requests refuse, before anything is enqueued (CPU: no call
here reaches a launch), and that their structures match the header."""
import ctypes
import os
import subprocess

import pytest
import torch

import bit_quantized_gemm_amd as w4

REACHED = (w4.OK, w4.EDEVICE, w4.ELAUNCH)   # checks passed; only the device check is left here


# ---------------------------------------------------------------- block_norm

def norm(**over):
    a = dict(x=0x10000000, y=0x20000000, gate=0x30000000, scale=0x31000000, shift=0x32000000, weight=0x33000000, bias=0x34000000,
             post_weight=0x35000000, out=0x40000000, residual=0x50000000, batch=2, tokens=7, width=100, x_stride=(700, 100),
             y_stride=(700, 100), gate_stride=(100, 0), scale_stride=(100, 0), shift_stride=(0, 0), out_stride=(700, 100),
             residual_stride=(700, 100), residual_scale=1.0, eps=1e-6, layer=1, post_norm=1, f16=0)
    a.update(over)
    return w4.block_norm_raw(w4.BlockNormArgs(*a.values()), 0)


NO_Y = dict(y=0, gate=0, residual=0, post_norm=0, post_weight=0)


@pytest.mark.parametrize("over,code", [
    (dict(batch=-1), "EINVAL"), (dict(tokens=-1), "EINVAL"), (dict(width=0), "EINVAL"), (dict(width=16385), "EINVAL"),
    (dict(f16=2), "EINVAL"), (dict(layer=2), "EINVAL"), (dict(post_norm=-1), "EINVAL"), (dict(eps=0.0), "EINVAL"),
    (dict(eps=-1e-6), "EINVAL"), (dict(eps=2.0), "EINVAL"), (dict(eps=float("nan")), "EINVAL"),
    (dict(residual_scale=float("inf")), "EINVAL"), (dict(residual_scale=float("nan")), "EINVAL"),
    (dict(batch=1 << 16, tokens=1 << 15), "EINVAL"), (dict(y=0), "EINVAL"), (dict(NO_Y, gate=0x30000000), "EINVAL"),
    (dict(NO_Y, residual=0x50000000), "EINVAL"), (dict(NO_Y, post_norm=1), "EINVAL"), (dict(NO_Y, residual_scale=2.0), "EINVAL"),
    (dict(post_norm=0), "EINVAL"), (dict(x_stride=(700, -100)), "EINVAL"), (dict(gate_stride=(1 << 61, 0)), "EINVAL"),
    (dict(out_stride=(700, 0)), "EINVAL"), (dict(out_stride=(0, 100)), "EINVAL"), (dict(residual_stride=(700, 99)), "EINVAL"),
    (dict(x=0), "EINVAL"), (dict(out=0), "EINVAL"), (dict(x=0x10000001), "EALIGN"), (dict(weight=0x33000001), "EALIGN"),
    (dict(residual=0x50000001), "EALIGN"), (dict(out=0x10000002), "EOVERLAP"), (dict(out=0x20000000, out_stride=(1400, 200)), "EOVERLAP"),
    (dict(residual=0x40000010), "EOVERLAP"), (dict(residual=0x40000000), "EOVERLAP"), (dict(gate=0x40000000), "EOVERLAP"),
    (dict(shift=0x50000100), "EOVERLAP"), (dict(weight=0x40000002), "EOVERLAP"), (dict(post_weight=0x50000002), "EOVERLAP")])
def test_norm_refuses(over, code):
    assert norm(**over) == getattr(w4, code)


@pytest.mark.parametrize("over", [
    dict(), NO_Y, dict(NO_Y, out=0x10000000), dict(out=0x10000000, residual=0x20000000), dict(residual=0x10000000),
    dict(residual=0), dict(gate=0, scale=0, shift=0, weight=0, bias=0, post_weight=0), dict(post_norm=0, post_weight=0),
    dict(x_stride=(0, 0)), dict(scale_stride=(700, 100)), dict(batch=1, out_stride=(0, 100)), dict(width=1, out_stride=(7, 1))])
def test_norm_accepts(over):
    assert norm(**over) in REACHED


def test_norm_empty_and_null():
    assert norm(batch=0) == w4.OK and norm(tokens=0, x=0, out=0) == w4.OK
    assert w4._native.load().block_norm(None, None) == w4.EINVAL


# ---------------------------------------------------------------- cache_append

def append(**over):
    a = dict(k=0x10000000, v=0x20000000, k_cache=0x30000000, v_cache=0x40000000, slots=0x50000000, tokens=10, heads=4, head_dim=64,
             pages=5, page_size=16, k_stride=(256, 64), v_stride=(256, 64), k_cache_stride=(4096, 256, 64), v_cache_stride=(4096, 256, 64))
    a.update(over)
    return w4.cache_append_raw(w4.CacheAppendArgs(*a.values()), 0)


ONE = dict(k_cache_stride=(8192, 256, 64), v_cache_stride=(8192, 256, 64))


@pytest.mark.parametrize("over,code", [
    (dict(tokens=-1), "EINVAL"), (dict(tokens=(1 << 30) + 1), "EINVAL"), (dict(heads=0), "EINVAL"), (dict(heads=1 << 20), "EINVAL"),
    (dict(head_dim=0), "EINVAL"), (dict(head_dim=12), "EINVAL"), (dict(head_dim=136), "EINVAL"), (dict(pages=-1), "EINVAL"),
    (dict(page_size=0), "EINVAL"), (dict(pages=1 << 20, page_size=1 << 11), "EINVAL"), (dict(k_stride=(256, -64)), "EINVAL"),
    (dict(v_stride=(260, 64)), "EINVAL"), (dict(k_cache_stride=(4096, 256, 32)), "EINVAL"), (dict(v_cache_stride=(0, 256, 64)), "EINVAL"),
    (dict(k_cache_stride=(4096, 260, 64)), "EINVAL"), (dict(k=0), "EINVAL"), (dict(v_cache=0), "EINVAL"), (dict(slots=0), "EINVAL"),
    (dict(k=0x10000008), "EALIGN"), (dict(v_cache=0x40000002), "EALIGN"), (dict(slots=0x50000004), "EALIGN"),
    (dict(k=0x30000010), "EOVERLAP"), (dict(slots=0x40000008), "EOVERLAP"), (dict(v_cache=0x30000000), "EOVERLAP"),
    (dict(v_cache=0x30000080), "EOVERLAP"), (dict(ONE, v_cache=0x30001000), "EOVERLAP"),
    (dict(v_cache=0x30002000, k_cache_stride=(8192, 256, 64), v_cache_stride=(8192, 512, 64)), "EOVERLAP")])
def test_append_refuses(over, code):
    assert append(**over) == getattr(w4, code)


@pytest.mark.parametrize("over", [
    dict(), dict(k_stride=(0, 0)), dict(v=0x10000000), dict(ONE, v_cache=0x30002000), dict(tokens=1, k_stride=(3, 64)),
    dict(page_size=1, k_cache_stride=(256, 7, 64), v_cache_stride=(256, 7, 64))])
def test_append_accepts(over):
    assert append(**over) in REACHED


def test_append_empty_and_null():
    assert append(tokens=0, k=0) == w4.OK and append(pages=0, k_cache=0, v_cache=0) == w4.OK
    assert w4._native.load().cache_append(None, None) == w4.EINVAL


# ---------------------------------------------------------------- lora_adapters

def adapt(**over):
    a = dict(x=0x10000000, y=0x20000000, down=0x30000000, up=0x40000000, out=0x50000000, adapter=0x60000000, scaling=0x61000000,
             ranks=0x62000000, rows=10, K=64, N=100, adapters=3, rank=16, x_stride=64, y_stride=100, out_stride=100, f16=0,
             workspace=0x70000000, workspace_bytes=1 << 20)
    a.update(over)
    return w4.LoraAdaptersArgs(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(rows=-1), "EINVAL"), (dict(rows=w4.LORA_ADAPTERS_MAX_ROWS + 1), "EINVAL"), (dict(K=0), "EINVAL"), (dict(K=60), "EINVAL"),
    (dict(N=0), "EINVAL"), (dict(N=(1 << 30) + 1), "EINVAL"), (dict(adapters=0), "EINVAL"), (dict(rank=0), "EINVAL"),
    (dict(rank=129), "EINVAL"), (dict(f16=2), "EINVAL"), (dict(x_stride=-64), "EINVAL"), (dict(x_stride=68), "EINVAL"),
    (dict(out_stride=99), "EINVAL"), (dict(out_stride=0), "EINVAL"), (dict(y_stride=1 << 61), "EINVAL"),
    (dict(adapters=2**31 - 1, rank=128, K=1 << 30), "EINVAL"), (dict(x=0), "EINVAL"), (dict(y=0), "EINVAL"), (dict(down=0), "EINVAL"),
    (dict(up=0), "EINVAL"), (dict(out=0), "EINVAL"), (dict(adapter=0), "EINVAL"), (dict(x=0x10000008), "EALIGN"),
    (dict(down=0x30000002), "EALIGN"), (dict(up=0x40000001), "EALIGN"), (dict(y=0x20000001), "EALIGN"), (dict(adapter=0x60000002), "EALIGN"),
    (dict(scaling=0x61000001), "EALIGN"), (dict(ranks=0x62000002), "EALIGN"), (dict(workspace=0), "ESCRATCH"),
    (dict(workspace_bytes=64), "ESCRATCH"), (dict(workspace=0x70000008), "EALIGN"), (dict(out=0x20000002), "EOVERLAP"),
    (dict(out=0x20000000, out_stride=104), "EOVERLAP"), (dict(out=0x10000000), "EOVERLAP"), (dict(out=0x30000100), "EOVERLAP"),
    (dict(up=0x50000000), "EOVERLAP"), (dict(adapter=0x50000010), "EOVERLAP"), (dict(workspace=0x10000000), "EOVERLAP"),
    (dict(workspace=0x50000000), "EOVERLAP"), (dict(scaling=0x70000000), "EOVERLAP")])
def test_adapters_refuse(over, code):
    assert w4.lora_adapters_raw(adapt(**over), 0) == getattr(w4, code)


@pytest.mark.parametrize("over", [
    dict(), dict(scaling=0, ranks=0), dict(out=0x20000000), dict(x_stride=0, y_stride=0), dict(rows=1, x_stride=3, out_stride=0),
    dict(y=0x20000002, up=0x40000002, out=0x50000002)])
def test_adapters_accept(over):
    assert w4.lora_adapters_raw(adapt(**over), 0) in REACHED


def test_adapters_empty_null_and_workspace():
    assert w4.lora_adapters_raw(adapt(rows=0, x=0, workspace=0), 0) == w4.OK
    lib = w4._native.load()
    assert lib.lora_adapters(None, None) == w4.EINVAL and lib.lora_adapters_workspace(None) == w4.EINVAL
    need = w4.lora_adapters_workspace
    assert need(adapt(K=60)) == w4.EINVAL and need(adapt(rows=0)) == 0
    assert need(adapt(rows=1000, rank=17)) >= 1000 * 32 * 4
    top = need(adapt(rows=w4.LORA_ADAPTERS_MAX_ROWS, rank=128, N=1 << 30, K=1 << 30))
    assert top >= w4.LORA_ADAPTERS_MAX_ROWS * 128 * 4


# ---------------------------------------------------------------- packed_attention

def packed(**over):
    a = dict(q=0x10000000, k=0x20000000, v=0x30000000, out=0x40000000, lse=0, starts=0x50000000, tokens=100, seqs=3, q_heads=4, kv_heads=2,
             head_dim=64, q_stride=(256, 64), k_stride=(128, 64), v_stride=(128, 64), out_stride=(256, 64), scale=0.125, causal=1, f16=0)
    a.update(over)
    return w4.packed_attention_raw(w4.PackedAttentionArgs(*a.values()), 0)


@pytest.mark.parametrize("over,code", [
    (dict(tokens=-1), "EINVAL"), (dict(seqs=-1), "EINVAL"), (dict(seqs=4097), "EINVAL"), (dict(tokens=1 << 22, q_heads=500, kv_heads=500, q_stride=(32000, 64), k_stride=(32000, 64), v_stride=(32000, 64), out_stride=(32000, 64), k=1 << 44, v=1 << 45, out=1 << 46, starts=1 << 47, seqs=4096), "EINVAL"), (dict(q_heads=-4), "EINVAL"),
    (dict(kv_heads=0), "EINVAL"), (dict(q_heads=5), "EINVAL"), (dict(head_dim=0), "EINVAL"), (dict(head_dim=60), "EINVAL"),
    (dict(head_dim=136), "EINVAL"), (dict(scale=0.0), "EINVAL"), (dict(scale=float("nan")), "EINVAL"), (dict(causal=2), "EINVAL"),
    (dict(f16=-1), "EINVAL"), (dict(tokens=1 << 29), "EINVAL"), (dict(q_heads=1 << 20, kv_heads=1 << 20), "EINVAL"),
    (dict(tokens=2**31 - 1024, q_heads=1, kv_heads=1 << 20), "EINVAL"), (dict(q_stride=(-256, 64)), "EINVAL"), (dict(q_stride=(260, 64)), "EINVAL"),
    (dict(k_stride=(1 << 23, 64)), "EINVAL"), (dict(v_stride=(56, 64)), "EINVAL"), (dict(v_stride=(0, 64)), "EINVAL"),
    (dict(out_stride=(256, 0)), "EINVAL"), (dict(out_stride=(192, 64)), "EINVAL"), (dict(q=0), "EINVAL"), (dict(v=0), "EINVAL"),
    (dict(out=0), "EINVAL"), (dict(starts=0), "EINVAL"), (dict(q=0x10000008), "EALIGN"), (dict(k=0x20000002), "EALIGN"),
    (dict(starts=0x50000002), "EALIGN"), (dict(lse=0x60000001), "EALIGN"), (dict(out=0x10000000), "EOVERLAP"), (dict(out=0x30000010), "EOVERLAP"),
    (dict(lse=0x40000100), "EOVERLAP"), (dict(starts=0x40000100), "EOVERLAP"), (dict(lse=0x20000000), "EOVERLAP")])
def test_packed_refuses(over, code):
    assert packed(**over) == getattr(w4, code)


@pytest.mark.parametrize("over", [
    dict(), dict(causal=0, lse=0x60000000), dict(k=0x30000000), dict(k_stride=(0, 0), v_stride=(64, 0)), dict(tokens=1, v_stride=(8, 64)),
    dict(seqs=4096)])
def test_packed_accepts(over):
    assert packed(**over) in REACHED


def test_packed_empty_and_null():
    assert packed(tokens=0, q=0) == w4.OK and packed(seqs=0, starts=0) == w4.OK and packed(q_heads=0) == w4.OK
    assert w4._native.load().packed_attention(None, None) == w4.EINVAL


# ---------------------------------------------------------------- paged_attention

def paged(**over):
    a = dict(q=0x10000000, k_cache=0x20000000, v_cache=0x30000000, out=0x40000000, lse=0, table=0x50000000, lens=0x51000000, batch=2, q_len=1,
             q_heads=4, kv_heads=2, head_dim=64, pages=9, page_size=16, table_width=4, q_stride=(256, 256, 64), k_stride=(2048, 128, 64),
             v_stride=(2048, 128, 64), out_stride=(256, 256, 64), table_stride=4, scale=0.125, f16=0, workspace=0, workspace_bytes=0)
    a.update(over)
    return w4.PagedAttentionArgs(*a.values())


CUT = dict(table_width=400)


@pytest.mark.parametrize("over,code", [
    (dict(batch=-1), "EINVAL"), (dict(q_len=-1), "EINVAL"), (dict(q_heads=-2), "EINVAL"), (dict(kv_heads=0), "EINVAL"), (dict(q_heads=5), "EINVAL"),
    (dict(head_dim=20), "EINVAL"), (dict(head_dim=136), "EINVAL"), (dict(pages=-1), "EINVAL"), (dict(page_size=0), "EINVAL"),
    (dict(page_size=8), "EINVAL"), (dict(page_size=24), "EINVAL"), (dict(table_width=-1), "EINVAL"), (dict(table_width=1 << 26), "EINVAL"),
    (dict(q_len=1 << 30), "EINVAL"), (dict(batch=1 << 24), "EINVAL"), (dict(scale=0.0), "EINVAL"), (dict(scale=float("inf")), "EINVAL"),
    (dict(q_len=1 << 28, q_heads=2, kv_heads=1, out=1 << 45, lens=1 << 46, table=1 << 47), "EINVAL"),
    (dict(f16=2), "EINVAL"), (dict(q_stride=(256, 256, -64)), "EINVAL"), (dict(q_stride=(250, 256, 64)), "EINVAL"), (dict(k_stride=(2048, 1 << 23, 64)), "EINVAL"),
    (dict(v_stride=(2048, 56, 64)), "EINVAL"), (dict(k_stride=(2050, 128, 64)), "EINVAL"), (dict(out_stride=(256, 256, 0)), "EINVAL"),
    (dict(out_stride=(128, 256, 64)), "EINVAL"), (dict(table_stride=-4), "EINVAL"), (dict(q=0), "EINVAL"), (dict(k_cache=0), "EINVAL"),
    (dict(table=0), "EINVAL"), (dict(lens=0), "EINVAL"), (dict(out=0), "EINVAL"), (dict(q=0x10000008), "EALIGN"), (dict(v_cache=0x30000002), "EALIGN"),
    (dict(table=0x50000002), "EALIGN"), (dict(lens=0x51000001), "EALIGN"), (dict(lse=0x60000002), "EALIGN"), (dict(out=0x10000010), "EOVERLAP"),
    (dict(out=0x20000010), "EOVERLAP"), (dict(table=0x40000010), "EOVERLAP"), (dict(lse=0x40000010), "EOVERLAP"), (dict(lse=0x51000000), "EOVERLAP"),
    (CUT, "ESCRATCH"), (dict(CUT, workspace=0x60000000, workspace_bytes=8), "ESCRATCH"), (dict(CUT, workspace=0x60000008, workspace_bytes=1 << 28), "EALIGN"),
    (dict(CUT, workspace=0x30000000, workspace_bytes=1 << 28), "EOVERLAP")])
def test_paged_refuses(over, code):
    assert w4.paged_attention_raw(paged(**over), 0) == getattr(w4, code)


@pytest.mark.parametrize("over", [
    dict(), dict(lse=0x60000000), dict(table_width=0, table=0, k_cache=0), dict(pages=0, v_cache=0), dict(k_cache=0x30000000), dict(table_stride=0),
    dict(CUT, workspace=0x60000000, workspace_bytes=1 << 28), dict(pages=1, k_stride=(3, 128, 64)), dict(page_size=48)])
def test_paged_accepts(over):
    assert w4.paged_attention_raw(paged(**over), 0) in REACHED


def test_paged_empty_null_and_workspace():
    run, need = w4.paged_attention_raw, w4.paged_attention_workspace
    assert run(paged(batch=0, q=0), 0) == w4.OK and run(paged(q_len=0), 0) == w4.OK and run(paged(q_heads=0), 0) == w4.OK
    lib = w4._native.load()
    assert lib.paged_attention(None, None) == w4.EINVAL and lib.paged_attention_workspace(None) == w4.EINVAL
    assert need(paged()) == 0 and need(paged(**CUT)) > 0 and need(paged(page_size=8)) == w4.EINVAL and need(paged(table_width=0)) == 0


@pytest.mark.parametrize("page", [16, 32, 48, 80, 112, 1008, 4112, 2**20 - 16, 2**29])
def test_page_of_a_key(page):
    """The multiplier by which the kernel divides, at every border, for keys below 2^31."""
    n = 4
    while 1 << n < page:
        n += 1
    magic = ((1 << (31 + n)) + page - 1) // page
    assert magic < 2**32
    keys = [k for m in list(range(0, 70)) + [2**31 // page // 3, 2**31 // page - 1, 2**31 // page] for k in (m * page - 1, m * page, m * page + page - 1)]
    for k in keys + [2**31 - 1]:
        if 0 <= k < 2**31:
            assert (k * magic >> 32) >> (n - 1) == k // page


# ---------------------------------------------------------------- the Python checks

def test_python_checks():
    bf, z = torch.bfloat16, torch.zeros
    with pytest.raises(TypeError):
        w4.block_norm(z(4, 32))
    with pytest.raises(ValueError):
        w4.block_norm(z(4, 32, dtype=bf))                              # not on a GPU
    with pytest.raises(ValueError):
        w4.cache_append(*(z(1, 1, 8, dtype=bf) for _ in range(4)), z(1, dtype=torch.int64))


STRUCTURES = {"block_norm_t": "BlockNormArgs", "lora_adapters_t": "LoraAdaptersArgs", "packed_attention_t": "PackedAttentionArgs",
              "paged_attention_t": "PagedAttentionArgs", "cache_append_t": "CacheAppendArgs"}


def test_structures_match_the_header(tmp_path):
    """Field offsets of the ctypes structures equal those a C compiler gives the header's."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    names = {t: getattr(w4, c) for t, c in STRUCTURES.items()}
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
