"""What the build compiles and links again, with stand-in compilers."""

import os
import stat
import sys
import time

import pytest

import block_scaled_precision_gemm_gb300 as bsmm
from block_scaled_precision_gemm_gb300 import _build

# writes its inputs' names and its own run's number to the file after -o, or fails as told
COMPILER = """#!{python}
import os, sys
here = os.path.dirname(os.path.abspath(__file__))
name = os.path.basename(__file__)
fails = os.path.join(here, name + ".fails")
if os.path.exists(fails) and open(fails).read() in sys.argv:
    open(sys.argv[sys.argv.index("-o") + 1], "w").write("half")
    sys.exit(1)
log = os.path.join(here, name + ".log")
open(log, "a").write(" ".join(sys.argv[1:]) + "\\n")
runs = len(open(log).readlines())
parts = [open(a).read() for a in sys.argv[1:] if a.endswith(".o") and "-c" not in sys.argv]
open(sys.argv[sys.argv.index("-o") + 1], "w").write(f"{{name}} {{runs}} " + " ".join(parts))
"""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    csrc, bin_ = tmp_path / "csrc", tmp_path / "bin"
    csrc.mkdir(), bin_.mkdir()
    for n in ("a.cu", "b.cu", "tensor_lists.cpp"):
        (csrc / n).write_text("source")
    for n in ("nvcc", "g++"):
        (bin_ / n).write_text(COMPILER.format(python=sys.executable))
        (bin_ / n).chmod(0o755 | stat.S_IXUSR)
    monkeypatch.setenv("NVCC", str(bin_ / "nvcc"))
    monkeypatch.setenv("CXX", str(bin_ / "g++"))
    monkeypatch.setattr(_build, "CSRC", str(csrc))
    monkeypatch.setattr(_build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(_build, "LISTS", str(tmp_path / "lists.so"))
    monkeypatch.setattr(_build, "_newest_header", lambda: 0.0)
    return tmp_path


def runs(tree, name):
    log = tree / "bin" / (name + ".log")
    return log.read_text().splitlines() if log.exists() else []


def newer(source, than):
    """The source a millisecond newer than what was made of it."""
    t = os.stat(than).st_mtime_ns + 10 ** 6
    os.utime(source, ns=(t, t))
    while time.time_ns() < t + 10 ** 7:
        time.sleep(0.001)


def test_nothing_is_built_twice(tree):
    _build.build()
    assert len(runs(tree, "nvcc")) == 3 and len(runs(tree, "g++")) == 1
    _build.build()
    assert len(runs(tree, "nvcc")) == 3 and len(runs(tree, "g++")) == 1
    (tree / "lib.so").unlink()
    _build.build()
    assert len(runs(tree, "nvcc")) == 4 and len(runs(tree, "g++")) == 1


@pytest.mark.parametrize("fails", ["g++", "link"])
def test_objects_of_a_build_that_failed_are_linked_by_the_next(tree, fails):
    _build.build()
    old = (tree / "lib.so").read_text()
    newer(tree / "csrc" / "a.cu", tree / "_build" / "a.cu.o")
    newer(tree / "csrc" / "tensor_lists.cpp", tree / "lists.so")
    if fails == "g++":
        (tree / "bin" / "g++.fails").write_text("-o")
        with pytest.raises(RuntimeError, match="failed for"):
            _build.build()
        (tree / "bin" / "g++.fails").unlink()
    else:  # the link of new objects never came about
        real = _build.subprocess.run
        _build.subprocess.run = lambda c, **kw: real(["false"] if "-shared" in c and c[0].endswith("nvcc") else c, **kw)
        try:
            with pytest.raises(RuntimeError, match="link failed"):
                _build.build()
        finally:
            _build.subprocess.run = real
    _build.build()
    assert (tree / "lib.so").read_text() != old


@pytest.mark.parametrize("word,tool,made", [("-c", "nvcc", "_build/a.cu.o"), ("-lcudart_static", "nvcc", "lib.so"),
                                            ("-o", "g++", "lists.so")])
def test_a_command_that_fails_leaves_what_was_there(tree, word, tool, made):
    _build.build()
    old = (tree / made).read_text()
    for n in ("a.cu", "tensor_lists.cpp"):
        newer(tree / "csrc" / n, tree / ("lists.so" if n.endswith("cpp") else "_build/a.cu.o"))
    (tree / "bin" / (tool + ".fails")).write_text(word)
    with pytest.raises(RuntimeError, match="failed"):
        _build.build()
    assert (tree / made).read_text() == old
    (tree / "bin" / (tool + ".fails")).unlink()
    _build.build()
    assert (tree / made).read_text() != old
    assert not [f for f in os.listdir(tree) + os.listdir(tree / "_build") if f.endswith(".part")]


@pytest.mark.parametrize("what", ["torch", "python"])
def test_another_torch_or_python_compiles_the_lists_again(tree, monkeypatch, what):
    import torch
    _build.build()
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    else:
        real = _build.sysconfig.get_config_var
        monkeypatch.setattr(_build.sysconfig, "get_config_var", lambda n: "cpython-0" if n == "SOABI" else real(n))
    _build.build()
    assert len(runs(tree, "g++")) == 2 and len(runs(tree, "nvcc")) == 3
    _build.build()
    assert len(runs(tree, "g++")) == 2


def test_lists_that_cannot_be_loaded_say_why(monkeypatch):
    monkeypatch.setattr(bsmm, "_LISTS", None)
    monkeypatch.delattr(bsmm, "_tensor_lists", raising=False)
    monkeypatch.setitem(sys.modules, "block_scaled_precision_gemm_gb300._tensor_lists", None)
    with pytest.raises(RuntimeError, match="cannot be loaded.*: .*halted"):
        bsmm._lists()
