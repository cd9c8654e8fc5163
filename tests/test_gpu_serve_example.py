"""The example that serves several requests at small sizes (MI355X): the operators together,
through their public entry points."""
import importlib.util
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
FOLDER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, FOLDER)
    spec = importlib.util.spec_from_file_location("serve_requests", os.path.join(FOLDER, "serve_requests.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("prompts,tokens,heads,kv_heads,page", [("70,1,129,33", 5, 4, 2, 16), ("200", 3, 2, 2, 64), ("3,5,1,1,40,64,2", 4, 6, 1, 32)])
def test_requests(example, prompts, tokens, heads, kv_heads, page):
    """Within 0.25 of what the block adds, against the plain block with the same 4-bit values: 16-bit
    roundings between the operators, and the codes that they move to the neighbouring value, at
    most a quarter (8 saturating at 6) of a block's largest magnitude each."""
    far = example.main(["--prompts", prompts, "--tokens", str(tokens), "--heads", str(heads), "--kv-heads", str(kv_heads), "--page", str(page),
                        "--steps", "2"])
    assert far < 0.25


def test_requests_do_not_meet(example):
    """A request's results with others beside it are those that it has alone, byte for byte, but for
    its residual's neighbours in the 4-bit layer's kernels, which depend on the number of rows."""
    block = example.Block(2, 1, 2)
    g = torch.Generator(device="cuda").manual_seed(3)
    a, b = (torch.randn(n, 256, generator=g, device="cuda").bfloat16() for n in (80, 112))
    which = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    both = block.prompts(torch.cat([a, b]), [80, 112], which, example.Cache(2, 128, 1, 128, 16, "cuda"))
    other = block.prompts(torch.cat([a, b * 3]), [80, 112], which, example.Cache(2, 128, 1, 128, 16, "cuda"))
    assert torch.equal(both[0][:80], other[0][:80]) and torch.equal(both[1][:80], other[1][:80])
    assert not torch.equal(both[1][80:], other[1][80:])
