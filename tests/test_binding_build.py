"""The CPython marshalling is built for the interpreter that loads it (no GPU needed)."""
import importlib
import importlib.machinery
import os

import pytest

import mixture_experts_grouped_align_gb300 as moe

b = importlib.import_module("mixture_experts_grouped_align_gb300.build")  # the package's `build` is its function


def test_the_file_names_its_interpreter():
    moe.build()
    assert b.BINDING.endswith(importlib.machinery.EXTENSION_SUFFIXES[0])
    assert os.path.exists(b.BINDING)


def test_another_interpreter_s_file_is_not_taken(monkeypatch, tmp_path):
    moe.build()
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_binding.cpython-399-none.so"))
    assert b.stale() == {b.BINDING}


def test_the_library_stands_without_the_binding(monkeypatch, tmp_path):
    """Where Python's headers are missing the calls without the binding still work; building says so."""
    lib = moe.build()
    before = os.path.getmtime(lib)
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(b, "python_include", lambda: str(tmp_path))
    with pytest.raises(RuntimeError, match="Python.h"):
        b.build()
    assert os.path.getmtime(lib) == before
