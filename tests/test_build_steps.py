"""The library and the torch binding are separate steps of the build: the library needs
nvcc alone.  Stand-ins for the compilers write empty outputs."""
import importlib.util
import os
import stat

import pytest

from stream_compaction_gb300 import build


def script(path, text):
    path.write_text("#!/bin/sh\n" + text)
    path.chmod(path.stat().st_mode | stat.S_IXUSR)
    return str(path)


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A package folder with one source of each kind, a stand-in nvcc, and a stand-in host compiler."""
    csrc, root = tmp_path / "pkg" / "csrc", tmp_path
    csrc.mkdir(parents=True)
    (root / "include").mkdir()
    for f in (csrc / "a.cu", csrc / "sc_bind.cpp", root / "include" / "sc_scan.h", root / "include" / "sc_seq.h"):
        f.write_text("")
    touch = 'while [ $# -gt 0 ]; do if [ "$1" = -o ]; then : > "$2"; fi; shift; done\n'
    monkeypatch.setenv("NVCC", script(tmp_path / "nvcc", touch))
    monkeypatch.setenv("CXX", script(tmp_path / "good", touch))
    monkeypatch.setattr(build, "CSRC", str(csrc))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "pkg" / "_build"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "pkg" / "libsc_gb300.so"))
    monkeypatch.setattr(build, "BIND", str(tmp_path / "pkg" / "_seqbind.so"))
    monkeypatch.setattr(build, "ROOT", str(root))
    return tmp_path


def without_torch(monkeypatch):
    found = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else found(name, *a))


def test_library_and_binding(tree):
    pytest.importorskip("torch")
    assert not build.up_to_date()
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and os.path.exists(build.BIND) and build.up_to_date()


def test_without_torch_the_library_is_built(tree, monkeypatch, capsys):
    without_torch(monkeypatch)
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.BIND)
    assert "torch" in capsys.readouterr().err
    assert build.up_to_date()  # there is nothing more to build here


def test_a_failing_binding_leaves_the_library(tree, monkeypatch):
    pytest.importorskip("torch")
    monkeypatch.setenv("CXX", script(tree / "bad", "echo no headers >&2; exit 1\n"))
    with pytest.raises(RuntimeError, match="no headers"):
        build.build()
    assert os.path.exists(build.LIB) and not build.up_to_date()
    monkeypatch.setenv("CXX", str(tree / "good"))
    before = os.stat(build.LIB).st_mtime_ns
    build.build()
    assert os.path.exists(build.BIND) and os.stat(build.LIB).st_mtime_ns == before  # only what was missing


def test_a_host_without_a_compiler_for_the_binding(tree, monkeypatch):
    pytest.importorskip("torch")
    monkeypatch.setenv("CXX", str(tree / "nowhere"))
    with pytest.raises(RuntimeError, match="binding"):
        build.build()
    assert os.path.exists(build.LIB)

def test_another_torch_rebuilds_the_binding(tree, monkeypatch):
    pytest.importorskip("torch")
    build.build()
    later = os.stat(build.BIND).st_mtime + 10
    version = tree / "torch" / "version.py"
    version.parent.mkdir()
    version.write_text("")
    (tree / "torch" / "__init__.py").write_text("")
    os.utime(version, (later, later))
    spec = importlib.util.spec_from_file_location("torch", tree / "torch" / "__init__.py")
    found = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: spec if name == "torch" else found(name, *a))
    assert not build.up_to_date()
