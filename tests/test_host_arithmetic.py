"""The host side of the operators for many requests at the ends of its integers (CPU): built for the
host alone with traps where a sum or product leaves its type, and called with sizes and strides
from all over their types. No code for a GPU is in that library; the calls end at their
checks or where they look for a device."""
import os
import re
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

from bit_quantized_gemm_amd import build as B

SOURCES = ("block_norm.hip", "cache_append.hip", "lora_adapters.hip", "packed_attention.hip", "paged_attention.hip")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CLANG = os.path.join(B.LLVM, "clang++")
TRAPS = ["-Xarch_host", "-fsanitize=signed-integer-overflow,integer-divide-by-zero,shift,bounds,float-cast-overflow",
         "-Xarch_host", "-fsanitize-trap=all"]
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up device addresses: needs a machine without a GPU")


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    d = tmp_path_factory.mktemp("host")

    def one(src):
        out = d / (src + ".o")
        flags = [f for f in B.compile_flags() if f not in ("-Xclang", "-target-feature", "-packed-fp32-ops")]
        subprocess.run([B.hipcc()] + flags + ["--offload-host-only"] + TRAPS + ["-c", os.path.join(B.CSRC, src), "-o", str(out)],
                       check=True, capture_output=True)
        return str(out)

    with ThreadPoolExecutor(5) as ex:
        objects = list(ex.map(one, SOURCES))
    # an empty bundle where each object expects its device code; no resources
    names = re.findall(r"U (__hip_fatbin_\w+)", subprocess.run(["nm", "-u"] + objects, check=True, capture_output=True, text=True).stdout)
    (d / "none.s").write_text('.section .hip_fatbin,"a"\n' + "".join(
        f'.globl {n}\n.p2align 12\n{n}:\n.ascii "__CLANG_OFFLOAD_BUNDLE__"\n.quad 0\n' for n in names))
    lib = d / "libhost.so"
    subprocess.run([CLANG, "-shared", "-fPIC", str(d / "none.s")] + objects + ["-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-ldl",
                                                                          "-o", str(lib)], check=True, capture_output=True)
    return str(lib)


CHILD = r"""
import ctypes, faulthandler, random, sys
import bit_quantized_gemm_amd as w4
name, lib, count = sys.argv[1], ctypes.CDLL(sys.argv[2]), int(sys.argv[3])
kind = {"block_norm": w4.BlockNormArgs, "cache_append": w4.CacheAppendArgs, "lora_adapters": w4.LoraAdaptersArgs,
        "packed_attention": w4.PackedAttentionArgs, "paged_attention": w4.PagedAttentionArgs}[name]
run = getattr(lib, name)
need = getattr(lib, name + "_workspace", None)
if need:
    need.restype = ctypes.c_int64
rng = random.Random(7)
INTS = [0, 1, 2, 3, 7, 8, 9, 15, 16, 17, 24, 32, 48, 63, 64, 65, 100, 127, 128, 129, 255, 256, 1000, 1024, 4095, 4096, 4097, 16384, 65535, 65536, 2**20 - 1,
        2**20, 2**23, 2**24 - 1, 2**24, 2**26, 2**28, 2**29, 2**30 - 1024, 2**30 - 1, 2**30, 2**30 + 1, 2**31 - 1025, 2**31 - 1024, 2**31 - 64, 2**31 - 1, -1, -2**31,
        3145728]
LONGS = [0, 8, 16, 64, 128, 4096, 2**20, 2**23 - 8, 2**23, 2**31, 2**32, 2**40, 2**58, 2**59, 2**60, 2**61, 2**62, 2**63 - 8, 2**63 - 1, -8, -2**63]
SMALL = {"heads": 8, "q_heads": 8, "kv_heads": 4, "head_dim": 64, "page_size": 16, "pages": 9, "table_width": 6, "batch": 3, "tokens": 50, "seqs": 3, "q_len": 2,
         "width": 100, "rows": 70, "K": 64, "N": 100, "adapters": 3, "rank": 16, "post_norm": 1}
codes, reached = {w4.OK, w4.EINVAL, w4.EALIGN, w4.EOVERLAP, w4.ESCRATCH, w4.EDEVICE, w4.ELAUNCH}, 0
for n in range(count):
    a, base = kind(), 1 << 40
    odd = {f for f, _ in kind._fields_ if rng.random() < rng.choice([0.05, 0.2, 0.5])}
    for f, t in kind._fields_:
        if t is ctypes.c_void_p:
            setattr(a, f, rng.choice([0, 2**64 - 16, 16, base + 2]) if f in odd and rng.random() < 0.2 else base)
            base += 1 << 44
        elif t is ctypes.c_int:
            setattr(a, f, rng.choice(INTS) if f in odd else SMALL.get(f, 0))
        elif t is ctypes.c_int64:
            setattr(a, f, rng.choice(LONGS) if f in odd else 2**50 if f == "workspace_bytes" else 2**13)
        elif t is ctypes.c_float:
            setattr(a, f, rng.choice([1.0, 0.0, 1e30, 1e-12, float("nan")]) if f in odd else 1e-3 if f != "residual_scale" else 1.0)
        else:
            size = t._length_
            for i in range(size):
                getattr(a, f)[i] = rng.choice(LONGS) if f in odd and rng.random() < 0.5 else (2**26, 2**16, 2**9)[i + 3 - size]
    said = {f: [*getattr(a, f)] if hasattr(getattr(a, f), "_length_") else getattr(a, f) for f, _ in kind._fields_}
    print(n, said, file=sys.stderr) if len(sys.argv) > 4 and n == int(sys.argv[4]) else None
    print(n, end=" ", flush=True)
    if need:
        need(ctypes.byref(a))
    code = run(ctypes.byref(a), None)
    assert code in codes, (code, said)
    reached += code in (w4.EDEVICE, w4.ELAUNCH)
print("reached", reached)
"""


@pytest.mark.parametrize("name", [s[:-4] for s in SOURCES])
def test_no_size_leaves_its_type(name, library):
    def child(*more):
        return subprocess.run([sys.executable, "-c", CHILD, name, library, "6000", *more], capture_output=True, text=True, cwd=ROOT, timeout=300)
    r = child()
    if r.returncode < 0:        # a trap: say which call
        n = r.stdout.split()[-1]
        pytest.fail(f"{name} ended with signal {-r.returncode} in call {child(n).stderr}")
    assert r.returncode == 0, r.stderr
    assert int(r.stdout.split()[-1]) > 300, r.stdout[-200:]      # calls that passed every check


def test_most_adapters(library):
    """As many adapters as an int holds, among the few rows' sizes."""
    code = ("import ctypes, sys, bit_quantized_gemm_amd as w4; f = ctypes.CDLL(sys.argv[1]).lora_adapters_workspace; f.restype = ctypes.c_int64;"
            "print(f(ctypes.byref(w4.LoraAdaptersArgs(rows=64, K=8, N=264, adapters=2**31 - 1, rank=1))))")
    r = subprocess.run([sys.executable, "-c", code, library], capture_output=True, text=True, cwd=ROOT, timeout=120)
    assert r.returncode == 0 and int(r.stdout) == 64 * 16 * 4, (r.returncode, r.stderr)
