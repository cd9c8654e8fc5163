"""The gfx950 assembly of the kernels for many requests (CPU: compiled, not run): as for the
block operators, no instruction but the direct-to-LDS loads' own sets or takes M0, nothing goes to
scratch memory, and float32 arithmetic is not packed."""
import os
import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from bit_quantized_gemm_amd import build as B
from test_block_asm import _instructions, m0_faults

SOURCES = ("block_norm.hip", "cache_append.hip", "lora_adapters.hip", "packed_attention.hip", "paged_attention.hip")


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    d = tmp_path_factory.mktemp("asm")

    def one(src):
        out = d / (src + ".s")
        flags = [f for f in B.compile_flags() if f != "-fPIC"]
        subprocess.run([B.hipcc()] + flags + ["--offload-device-only", "-S", os.path.join(B.CSRC, src), "-o", str(out)],
                       check=True, capture_output=True)
        return out.read_text()

    with ThreadPoolExecutor(5) as ex:
        return dict(zip(SOURCES, ex.map(one, SOURCES)))


@pytest.mark.parametrize("src", SOURCES)
def test_m0_is_only_the_loads(asm, src):
    code = _instructions(asm[src])
    assert not m0_faults(code), m0_faults(code)[:5]
    assert any(line.endswith(" lds") for line in code) == (src in ("packed_attention.hip", "paged_attention.hip"))


@pytest.mark.parametrize("src", SOURCES)
def test_no_scratch_and_no_packed_float32(asm, src):
    code = _instructions(asm[src])
    assert not [c for c in code if c.startswith(("scratch_", "v_pk_add_f32", "v_pk_mul_f32", "v_pk_fma_f32"))]
    assert set(re.findall(r"; ScratchSize: (\d+)", asm[src])) == {"0"}


def late_registers(code):
    """Buffer loads less than five wait states behind a lane read into their descriptor (the instruction set asks
    for five between a vector instruction's write of a scalar register and a memory instruction that takes it)."""
    bad = []
    for i, line in enumerate(code):
        m = re.match(r"^buffer_load\S* v\S+, (?:v\S+, )?s\[(\d+):(\d+)\]", line)
        states = 0
        for before in reversed(code[max(0, i - 6):i] if m else []):
            w = re.match(r"^v_read(?:first)?lane_b32 s(\d+),", before)
            if states < 5 and w and int(m[1]) <= int(w[1]) <= int(m[2]):
                bad.append((before, line, states))
            nop = re.match(r"^s_nop (\d+)", before)
            states += int(nop[1]) + 1 if nop else 1
    return bad


def test_late_registers_are_seen():
    load = "buffer_load_dwordx4 v1, s[4:7], 0 offen lds"
    late = ["v_readfirstlane_b32 s5, v2", "s_mov_b32 m0, s1", "s_nop 0", load]
    assert late_registers(late) and not late_registers(["v_readlane_b32 s8, v2, 3"] + late[1:])
    assert not late_registers([late[0], "s_nop 2"] + late[1:]) and late_registers([late[0], "s_nop 1"] + late[1:])


@pytest.mark.parametrize("src", ("attention.hip", "mxfp4_producer.hip", "packed_attention.hip", "paged_attention.hip"))
def test_loads_wait_for_their_descriptors(src, asm, tmp_path):
    text = asm.get(src)
    if text is None:
        out = tmp_path / "out.s"
        flags = [f for f in B.compile_flags() if f != "-fPIC"]
        subprocess.run([B.hipcc()] + flags + ["--offload-device-only", "-S", os.path.join(B.CSRC, src), "-o", str(out)],
                       check=True, capture_output=True)
        text = out.read_text()
    code = _instructions(text)
    assert any(line.startswith("buffer_load") for line in code)
    assert not late_registers(code), late_registers(code)[:5]
