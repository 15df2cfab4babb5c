"""CPU tests of the build: the library does not wait for the binding, and each is made again
when what it was made from or for has changed.  The compilers are stood in for."""
import importlib.metadata
import os
import subprocess
from types import SimpleNamespace

import pytest
import torch

from differential_attention_fwd_gb300 import _paged
from differential_attention_fwd_gb300 import build as build_mod


@pytest.fixture
def fake(tmp_path, monkeypatch):
    """A build into tmp_path whose commands only make their outputs; a list of them, as
    (what, output's name), and a set of words that make a command fail."""
    f = SimpleNamespace(ran=[], fail=set(), lib=str(tmp_path / "lib.so"), binding=str(tmp_path / "binding.so"))

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        f.ran.append(os.path.basename(out))
        bad = any(w in arg for w in f.fail for arg in cmd)
        if not bad:
            with open(out, "w"):
                pass
        return subprocess.CompletedProcess(cmd, int(bad), "", "stood in for")

    monkeypatch.setattr(build_mod.subprocess, "run", run)
    monkeypatch.setitem(build_mod.VARIANTS, None, (f.lib, str(tmp_path / "obj"), []))
    monkeypatch.setattr(build_mod, "BUILD", str(tmp_path / "obj"))
    monkeypatch.setattr(build_mod, "BINDING", f.binding)
    return f


def test_a_binding_that_fails_leaves_the_library(fake):
    for word in ("binding.cpp", "-ltorch_python"):      # its compiler, its linker
        fake.fail = {word}
        with pytest.raises(RuntimeError, match="binding"):
            build_mod.build()
        assert os.path.exists(fake.lib) and not os.path.exists(fake.binding)
        os.remove(fake.lib)


def test_a_library_that_fails_is_an_error(fake):
    fake.fail = {"paged.cu"}
    with pytest.raises(RuntimeError, match="nvcc"):
        build_mod.build()
    assert not os.path.exists(fake.lib)


def test_only_what_is_stale_is_made(fake):
    build_mod.build()
    assert {"binding.cpp.o", "rotary.cu.o", "lib.so.tmp", "binding.so.tmp"} <= set(fake.ran)
    fake.ran.clear()
    build_mod.build()
    assert fake.ran == []
    os.remove(fake.lib)
    build_mod.build()
    assert "lib.so.tmp" in fake.ran and "rotary.cu.o" in fake.ran and "binding.cpp.o" not in fake.ran
    fake.ran.clear()
    os.remove(fake.binding)
    build_mod.build()
    assert fake.ran == ["binding.cpp.o", "binding.so.tmp"]
    build_mod.build(force=True)
    assert {"rotary.cu.o", "lib.so.tmp"} <= set(fake.ran)


def test_another_torch_makes_the_binding_again(fake, monkeypatch):
    build_mod.build()
    fake.ran.clear()
    monkeypatch.setattr(build_mod, "torch_version", lambda: "1.0")
    build_mod.build()
    assert fake.ran == ["binding.cpp.o", "binding.so.tmp"]
    build_mod.build()
    assert len(fake.ran) == 2


def test_the_torch_that_imports_decides(monkeypatch):
    """Not what a package index knows of it, which may know nothing."""
    def unknown(name):
        raise importlib.metadata.PackageNotFoundError(name)
    monkeypatch.setattr(importlib.metadata, "version", unknown)
    assert build_mod.torch_version() == str(torch.__version__)


def test_a_binding_for_another_torch_is_not_loaded(monkeypatch):
    build_mod.build()
    monkeypatch.setattr(_paged, "_native", None)
    monkeypatch.setattr(build_mod, "torch_version", lambda: "1.0")
    with pytest.raises(RuntimeError, match="build it again"):
        _paged._load()
    monkeypatch.undo()
    assert _paged._load() is not None
