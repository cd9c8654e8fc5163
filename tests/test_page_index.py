"""The page of a key as paged_attention works it out (CPU: a host program built from the header that
the library's host side and kernels use)."""
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_quantized_gemm_amd", "csrc")
SOURCE = """
#include <stdio.h>
#include "w4a4_page_index.hpp"
static_assert(w4a4::page_index(48).of(47) == 0 && w4a4::page_index(48).of(48) == 1);
int main() {
  int page, key;
  while (scanf("%d %d", &page, &key) == 2) printf("%d\\n", w4a4::page_index(page).of(key));
}
"""
SIZES = sorted({16 * m for m in list(range(1, 66)) + [125, 127, 129, 257, 4095, 4096, 4097, 65535, 65537, 2**20 - 1, 2**22 + 1, 2**25 - 1]} |
               {2**n for n in range(4, 31)} | {2**n + 16 for n in range(4, 30)} | {2**n - 16 for n in range(5, 31)})


@pytest.fixture(scope="module")
def place_of(tmp_path_factory):
    d = tmp_path_factory.mktemp("page_index")
    (d / "t.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++20", "-O1", "-Wall", "-Wextra", "-Werror", f"-I{CSRC}", str(d / "t.cpp"), "-o", str(d / "t")], check=True)

    def run(pairs):
        text = "".join(f"{page} {key}\n" for page, key in pairs)
        return [int(x) for x in subprocess.run([str(d / "t")], input=text, capture_output=True, text=True, check=True).stdout.split()]
    return run


def test_every_border(place_of):
    """Both sides of the first borders, of some in the middle and of the last ones below 2^31."""
    pairs = []
    for page in SIZES:
        last = (2**31 - 1) // page
        pages = set(range(70)) | {last // 3, last // 2, last - 1, last, last + 1} | {2**k for k in range(31)} | {2**k - 1 for k in range(31)}
        keys = {0, 2**31 - 1, 2**30, 2**30 - 1} | {m * page + d for m in pages for d in (-1, 0, 1, page - 1)}
        pairs += [(page, k) for k in sorted(keys) if 0 <= k < 2**31]
    got = place_of(pairs)
    assert len(got) == len(pairs)
    wrong = [(pair, g) for pair, g in zip(pairs, got) if g != pair[1] // pair[0]]
    assert not wrong, wrong[:5]


def test_the_library_uses_it():
    """The multiplier is made and used in that header alone."""
    host = open(os.path.join(CSRC, "paged_attention.hip")).read()
    kernels = open(os.path.join(CSRC, "w4a4_attention.hpp")).read()
    assert "p.page_index = page_index(a->page_size);" in host and "return p.page_index.of(key);" in kernels
    assert "magic" not in host + kernels
