"""The in-tree build: what it links when.  The compilers are replaced; no GPU, no nvcc."""
import os
import subprocess
import sys

import pytest

from int8_kv_cache_gb300 import build as B


class Compilers:
    """Stands in for nvcc and g++: writes the output file, or fails where told to."""

    def __init__(self):
        self.ran = []
        self.fail = lambda cmd: False

    def __call__(self, cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        self.ran.append(os.path.basename(out).replace(".tmp", ""))
        if self.fail(cmd):
            return subprocess.CompletedProcess(cmd, 1, "", "refused")
        with open(out, "w") as f:
            f.write(" ".join(cmd))
        return subprocess.CompletedProcess(cmd, 0, "", "")


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A package of one kernel file and the binding, in a folder of its own."""
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    (csrc / "a.cu").write_text("1")
    (csrc / "binding.cpp").write_text("1")
    (tmp_path / "h.h").write_text("1")
    c = Compilers()
    for name, value in dict(PKG=str(tmp_path), CSRC=str(csrc), BUILD=str(tmp_path / "_build"),
                            LIB=str(tmp_path / "libint8kv.so"), HEADER=str(tmp_path / "h.h"),
                            BINDING=str(tmp_path / "_binding.so"), nvcc=lambda: "/usr/local/cuda/bin/nvcc").items():
        monkeypatch.setattr(B, name, value)
    monkeypatch.setattr(B.subprocess, "run", c)
    return tmp_path, c


def test_nothing_changed_nothing_compiled(tree):
    path, c = tree
    B.build()
    assert {"a.o", "binding.o", "libint8kv.so", "_binding.so"} <= set(c.ran)
    c.ran.clear()
    B.build()
    assert not {"a.o", "binding.o"} & set(c.ran)


@pytest.mark.parametrize("broken", ["a.o", "libint8kv.so.tmp", "_binding.so.tmp"])
def test_a_binding_of_another_header_is_never_kept(tree, broken):
    # a build that compiles the binding and fails at something else, then one that succeeds
    path, c = tree
    B.build()
    (path / "h.h").write_text("2")
    old = (path / "_binding.so").read_text()
    (path / "_binding.so").write_text("stale")
    c.fail = lambda cmd: cmd[cmd.index("-o") + 1].endswith(broken)
    with pytest.raises(RuntimeError):
        B.build()
    c.fail = lambda cmd: False
    B.build()
    assert (path / "_binding.so").read_text() == old


def test_the_library_does_not_wait_for_the_binding(tree):
    # a binding that does not compile is an error, with the library there for callers in C
    path, c = tree
    c.fail = lambda cmd: cmd[cmd.index("-o") + 1].endswith("binding.o")
    with pytest.raises(RuntimeError):
        B.build()
    assert (path / "libint8kv.so").exists()


def test_the_library_needs_no_pytorch(tree, monkeypatch):
    path, c = tree
    monkeypatch.setitem(sys.modules, "torch", None)
    assert B.build() == str(path / "libint8kv.so")
    assert (path / "libint8kv.so").exists() and not (path / "_binding.so").exists()
