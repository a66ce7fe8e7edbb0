"""The in-tree build (CPU only): the library does not need Python's headers, and the binding's compiled module is named
for the interpreter that it was built for."""
import importlib.machinery
import os
import sysconfig

import pytest

import rotated_w4a8_int8_gb300 as cr
from rotated_w4a8_int8_gb300 import _build

FAKE_NVCC = """#!/bin/sh
while [ $# -gt 0 ]; do [ "$1" = "-o" ] && touch "$2"; shift; done
"""


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """The build with its outputs in tmp_path, no sources and a compiler that only makes files."""
    nvcc = tmp_path / "nvcc"
    nvcc.write_text(FAKE_NVCC)
    nvcc.chmod(0o755)
    monkeypatch.setattr(_build, "nvcc", lambda: str(nvcc))
    monkeypatch.setattr(_build, "SOURCES", [("api.cu", "api", [])])
    for name in ("BUILD", "LIB", "MARSHAL"):
        monkeypatch.setattr(_build, name, str(tmp_path / os.path.basename(getattr(_build, name))))
    return tmp_path


def test_library_without_python_headers(elsewhere, monkeypatch, capfd):
    empty = elsewhere / "include"
    empty.mkdir()
    monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **k: {"include": str(empty), "platinclude": str(empty)})
    assert _build.build(force=True) == _build.LIB and os.path.exists(_build.LIB)
    assert not os.path.exists(_build.MARSHAL)
    assert "Python.h" in capfd.readouterr().err
    stamp = os.path.getmtime(_build.LIB)
    assert _build.build() == _build.LIB and os.path.getmtime(_build.LIB) == stamp      # nothing left to do


def test_module_is_built_where_headers_are(elsewhere):
    _build.build(force=True)
    assert os.path.exists(_build.MARSHAL)


def test_module_is_tagged_for_the_interpreter():
    suffix = importlib.machinery.EXTENSION_SUFFIXES[0]
    assert suffix != ".so" and os.path.basename(_build.MARSHAL) == "_marshal" + suffix
    _build.build()
    assert cr._operators().__file__ == _build.MARSHAL
