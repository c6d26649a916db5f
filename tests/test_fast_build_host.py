"""Building and choosing the extension module (no GPU)."""
import os
import subprocess

import pytest
import torch

from reciprocal_nearest_neighbour_b200 import _lib, build as rnn_build


@pytest.fixture
def compilers(monkeypatch, tmp_path):
    """Both compilers replaced: each writes its output, or fails.  The names of what ran."""
    ran, broken = [], set()

    def check_call(cmd):
        kind = "library" if rnn_build.LIB in cmd[-1] else "module"
        ran.append(kind)
        if kind in broken:
            raise FileNotFoundError(cmd[0]) if cmd[0] == "missing" else \
                subprocess.CalledProcessError(1, cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(kind)

    monkeypatch.setattr(rnn_build, "PKG", str(tmp_path))
    monkeypatch.setattr(rnn_build, "LIB", str(tmp_path / "librnn.so"))
    monkeypatch.setattr(rnn_build.subprocess, "check_call", check_call)
    return ran, broken


@pytest.mark.parametrize("cxx", ["g++", "missing"])
def test_the_library_is_built_without_the_module(compilers, monkeypatch, capfd, cxx):
    """No compiler for C++, or headers that do not fit: the library needs neither."""
    ran, broken = compilers
    broken.add("module")
    monkeypatch.setenv("CXX", cxx)
    assert rnn_build.build() == rnn_build.LIB and os.path.exists(rnn_build.LIB)
    assert ran == ["library", "module"]
    assert "without the extension module" in capfd.readouterr().err
    with pytest.raises((subprocess.CalledProcessError, OSError)):
        rnn_build.build_fast()


def test_a_library_that_does_not_build_is_an_error(compilers):
    ran, broken = compilers
    broken.add("library")
    with pytest.raises(subprocess.CalledProcessError):
        rnn_build.build()
    assert ran == ["library"]


def test_a_module_of_other_sources_does_not_stay(compilers):
    """Where it cannot be built again it may not fit the library."""
    ran, broken = compilers
    old = rnn_build.build_fast()
    os.utime(old, (1, 1))
    broken.add("module")
    rnn_build.build()
    assert not os.path.exists(old)
    broken.clear()
    new = rnn_build.build_fast()
    broken.add("module")
    rnn_build.build(force=True)          # of these sources: it stays
    assert os.path.exists(new)


def test_another_torch_needs_another_module(compilers, monkeypatch):
    """The file's name says what it was built for, so one for another torch or Python is
    neither kept nor loaded."""
    ran, _ = compilers
    first = rnn_build.build_fast()
    assert ran == ["module"] and rnn_build.build_fast() == first and ran == ["module"]
    monkeypatch.setattr(torch, "__version__", "9.9.0+cu999")
    second = rnn_build.build_fast()
    assert second != first and ran == ["module", "module"]
    assert os.path.exists(first) and os.path.exists(second)


def test_no_module_for_this_torch_means_the_python_forms(monkeypatch):
    monkeypatch.setattr(_lib, "fast", None)
    monkeypatch.setattr(torch, "__version__", "9.9.0+cu999")
    assert _lib.load_fast() is _lib._Python


def test_the_module_of_this_torch_is_loaded(monkeypatch):
    rnn_build.build()
    rnn_build.build_fast()
    monkeypatch.setattr(_lib, "fast", None)
    module = _lib.load_fast()
    assert module.__name__.endswith("_fast") and module.__file__ == rnn_build.fast_path()
    assert _lib.load_fast() is module
