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
