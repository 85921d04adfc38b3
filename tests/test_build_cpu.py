"""The build's order and its idea of what is out of date, with the compilers
and linkers replaced by stand-ins that write small files."""
import importlib.metadata
import importlib.util
import os

import pytest

from row_normalization_inner_gb300 import build


@pytest.fixture
def made(tmp_path, monkeypatch):
    """What the last builds compiled and linked, in order."""
    log = []

    def compile_one(src):
        log.append(os.path.basename(src))
        return str(tmp_path / "x.o"), "log"

    def compile_tensors():
        log.append("tensors.cpp")
        return str(tmp_path / "tensors.o")

    def link(cmd, out):
        log.append(os.path.basename(out))
        with open(out, "w") as f:
            f.write("linked")

    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libnf.so"))
    monkeypatch.setattr(build, "TENSORS", str(tmp_path / "_tensors.so"))
    monkeypatch.setattr(build, "_compile", compile_one)
    monkeypatch.setattr(build, "_compile_tensors", compile_tensors)
    monkeypatch.setattr(build, "_link", link)
    return log


def test_both_libraries_once(made):
    build.build()
    assert "libnf.so" in made and "_tensors.so" in made and "k_embed.cu" in made
    made.clear()
    assert build.build() == build.LIB and made == []


def test_the_c_library_needs_no_pytorch(made, monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.TENSORS)
    made.clear()
    build.build()  # nothing is out of date
    assert made == []


def test_the_c_library_is_there_where_the_helpers_do_not_compile(made, monkeypatch):
    def fails():
        raise RuntimeError("no Python.h")
    monkeypatch.setattr(build, "_compile_tensors", fails)
    with pytest.raises(RuntimeError, match="Python.h"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.TENSORS)


def test_another_pytorch_rebuilds_the_helpers_alone(made, monkeypatch):
    build.build()
    made.clear()
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "0.0.other")
    build.build()
    assert made == ["tensors.cpp", "_tensors.so"]
    made.clear()
    build.build()
    assert made == []
