"""The C library builds where torch or Python's headers are missing; the binding is left
out with a message, and built where both are there (CPU: the compiler steps are recorded, not
run)."""
import importlib.util
import os
import sys
import sysconfig

import pytest

from bit_quantized_gemm_amd import build as B


@pytest.fixture
def steps(monkeypatch, tmp_path):
    done = []
    monkeypatch.setattr(B, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(B, "_build_one", lambda path, *a: done.append(path))
    monkeypatch.setattr(B, "_run", lambda cmd, verbose: done.append(cmd[cmd.index("-o") + 1]))
    monkeypatch.setattr(os, "replace", lambda a, b: None)
    return done


def test_everything_here(steps, capsys):
    assert B.build() == B.LIB_PATH
    assert steps == list(B.LIBS) + [B.BINDING_PATH + ".tmp"] and not capsys.readouterr().err


def test_without_torch(steps, monkeypatch, capsys):
    found = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name.split(".")[0] == "torch" else found(name, *a))
    # importing torch would raise there
    monkeypatch.setitem(sys.modules, "torch.utils.cpp_extension", None)
    assert B.build() == B.LIB_PATH
    assert steps == list(B.LIBS)
    assert "torch is missing" in capsys.readouterr().err


def test_without_python_headers(steps, monkeypatch, capsys, tmp_path):
    paths = dict(sysconfig.get_paths(), include=str(tmp_path))
    monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **k: paths)
    assert B.build() == B.LIB_PATH
    assert steps == list(B.LIBS)
    assert "Python.h is missing" in capsys.readouterr().err
