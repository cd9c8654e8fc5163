"""Tests that hand made-up device addresses to calls which pass every check (CPU): on a
machine with a GPU they would launch kernels on those addresses, so they are skipped there."""
import ast
import os

import pytest
import torch

import conftest

HERE = os.path.dirname(os.path.abspath(__file__))


class Item:
    def __init__(self, file, name, keywords=()):
        self.fspath, self.name, self.keywords, self.marks = os.path.join(HERE, file), name, keywords, []

    def add_marker(self, mark):
        self.marks.append(mark.name)


@pytest.mark.parametrize("gpu", [True, False])
def test_skipped_where_a_gpu_is(gpu, monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_available", lambda: gpu)
    risky = [Item(f, n + "[x0]") for f, names in conftest.MADE_UP_ADDRESSES.items() for n in names]
    others = [Item("test_block_refusals.py", "test_rotary_refuses[over0-EINVAL]"), Item("test_abi.py", "test_quantize_overlap")]
    on_gpu = [Item("test_gpu_few.py", "test_sizes", ("gpu",))]
    conftest.pytest_collection_modifyitems(None, risky + others + on_gpu)
    assert all(i.marks == (["skip"] if gpu else []) for i in risky)
    assert not any(i.marks for i in others)
    assert all(i.marks == ([] if gpu else ["skip"]) for i in on_gpu)


def _passes_the_checks(fn):
    """Whether a test expects a code that only a call past all checks gives."""
    for node in ast.walk(fn):
        if isinstance(node, ast.Compare) and any(isinstance(op, ast.In) for op in node.ops):
            text = ast.unparse(node.comparators[0])
            if text == "REACHED" or "EDEVICE" in text:
                return True
    return False


def test_the_list_is_complete():
    found = {}
    for name in sorted(os.listdir(HERE)):
        if not (name.startswith("test_") and name.endswith(".py")):
            continue
        tree = ast.parse(open(os.path.join(HERE, name)).read())
        tests = {f.name for f in tree.body if isinstance(f, ast.FunctionDef) and f.name.startswith("test_") and _passes_the_checks(f)}
        if tests:
            found[name] = tests
    assert found == conftest.MADE_UP_ADDRESSES
