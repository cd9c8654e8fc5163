"""The transformer block example at small sizes (MI355X): the operators together,
through their public entry points."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "transformer_block.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("transformer_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("batch,height,width,text,heads", [(1, 16, 16, 77, 2), (3, 9, 7, 33, 1), (2, 20, 13, 300, 3)])
def test_block(example, batch, height, width, text, heads):
    """Within 0.25 of what the block adds, against the plain block with the same 4-bit
    values: 16-bit roundings between the operators, and the codes that they move to
    the neighbouring value, at most a quarter (8 saturating at 6) of a block's
    largest magnitude each."""
    far = example.main(["--batch", str(batch), "--height", str(height), "--width", str(width), "--text", str(text),
                        "--heads", str(heads), "--steps", "2"])
    assert far < 0.25


def test_no_text_at_all(example):
    """A sequence whose text has no states attends to the image alone."""
    block = example.Block(2)
    x, vec, text, lens, pos = example.inputs(2, 8, 8, 40, 256)
    lens[1] = 0
    y = block(x, vec, text, lens, pos)
    text[1] = float("inf")                       # never read past its length
    again = block(x, vec, text.nan_to_num(posinf=7.0), lens, pos)
    assert torch.isfinite(y).all() and torch.equal(y[1], again[1])
