"""The gfx950 assembly of the block operators' kernels (CPU: compiled, not run).

Their direct-to-LDS loads set M0 in inline assembly, which the compiler does not see:
it reserves M0 and would keep a value of its own in it across such a load, or take ours.
So no other instruction of these kernels may set or take M0. Beside that: no spills to
scratch, and no packed float32 arithmetic.
"""
import os
import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from bit_quantized_gemm_amd import build as B

SOURCES = ("attention.hip", "mxfp4_producer.hip", "mxfp4_few.hip", "rotary.hip")
# instructions that take M0 without naming it
HIDDEN_M0 = re.compile(r"^(v_movrel|s_movrel|v_interp|s_sendmsg|ds_gws|ds_\w*addtid|ds_ordered|s_ttrace|global_load_lds)")


def _instructions(text):
    """Instruction lines without comments, labels and directives."""
    out = []
    for line in text.splitlines():
        body = line.split(";")[0].strip()
        if body and not body.startswith(".") and not body.endswith(":"):
            out.append(re.sub(r"\s+", " ", body))
    return out


def m0_faults(code):
    """What breaks the rule: every mention of M0 belongs to `s_mov_b32 m0, sN; s_nop 0;
    buffer_load_dwordx4 ... lds`, every load to LDS to such a group, nothing takes M0 unseen."""
    bad, covered = [], set()
    for i, line in enumerate(code):
        if re.search(r"\bm0\b", line):
            group = code[i:i + 3]
            if re.match(r"^s_mov_b32 m0, s\d+$", line) and len(group) == 3 and group[1] == "s_nop 0" and \
                    re.match(r"^buffer_load_dwordx4 v\d+, s\[\d+:\d+\], 0 offen lds$", group[2]):
                covered.add(i + 2)
            else:
                bad.append(line)
        elif HIDDEN_M0.match(line):
            bad.append(line)
    bad += [line for i, line in enumerate(code) if re.search(r"\blds$", line) and i not in covered]
    return bad


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    d = tmp_path_factory.mktemp("asm")

    def one(src):
        out = d / (src + ".s")
        flags = [f for f in B.compile_flags() if f != "-fPIC"]
        subprocess.run([B.hipcc()] + flags + ["--offload-device-only", "-S", os.path.join(B.CSRC, src), "-o", str(out)],
                       check=True, capture_output=True)
        return out.read_text()

    with ThreadPoolExecutor(4) as ex:
        return dict(zip(SOURCES, ex.map(one, SOURCES)))


@pytest.mark.parametrize("src", SOURCES)
def test_m0_is_only_the_loads(asm, src):
    code = _instructions(asm[src])
    assert len(code) > 1000
    assert not m0_faults(code), m0_faults(code)[:5]
    loads = sum(line.endswith(" lds") for line in code)
    assert (loads > 0) == (src in ("attention.hip", "mxfp4_producer.hip"))


@pytest.mark.parametrize("src", SOURCES)
def test_no_scratch_and_no_packed_float32(asm, src):
    code = _instructions(asm[src])
    assert not [c for c in code if c.startswith(("scratch_", "v_pk_add_f32", "v_pk_mul_f32", "v_pk_fma_f32"))]
    assert set(re.findall(r"; ScratchSize: (\d+)", asm[src])) == {"0"}


@pytest.mark.parametrize("plant", ["s_mov_b32 m0, -1", "s_add_u32 m0, s4, 16", "v_movrels_b32_e32 v1, v2", "s_mov_b32 s3, m0",
                                   "buffer_load_dwordx4 v1, s[4:7], 0 offen lds", "s_sendmsg sendmsg(MSG_INTERRUPT)"])
def test_the_rule_sees_what_breaks_it(plant):
    good = ["v_add_u32_e32 v0, v1, v2", "s_mov_b32 m0, s9", "s_nop 0", "buffer_load_dwordx4 v7, s[12:15], 0 offen lds", "s_endpgm"]
    assert not m0_faults(good)
    for at in range(len(good) + 1):
        assert m0_faults(good[:at] + [plant] + good[at:])
