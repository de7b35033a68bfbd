"""What the build does where the extension module of the serving calls cannot be
made: compilers are stand-ins here, so that nothing is compiled."""
import os
import subprocess
import sys

import pytest

from block_sparse_compressed_gb300 import build as B


@pytest.fixture
def place(tmp_path, monkeypatch):
    """A package folder of its own and a record of the commands run."""
    csrc, inc = tmp_path / "pkg" / "csrc", tmp_path / "include"
    csrc.mkdir(parents=True)
    inc.mkdir()
    for f in ("a.cu", "b.cu", "hca_py.cpp"):
        (csrc / f).write_text("//\n")
    (inc / "hca.h").write_text("//\n")
    pkg = str(tmp_path / "pkg")
    monkeypatch.setattr(B, "HERE", pkg)
    monkeypatch.setattr(B, "CSRC", str(csrc))
    monkeypatch.setattr(B, "BUILD", os.path.join(pkg, "_build"))
    monkeypatch.setattr(B, "LIB", os.path.join(pkg, "libhca.so"))
    monkeypatch.setattr(B, "PY_LIB", os.path.join(pkg, os.path.basename(B.PY_LIB)))
    monkeypatch.setattr(B, "_nvcc", lambda: "/opt/cuda/bin/nvcc")
    monkeypatch.delenv("CXX", raising=False)
    ran = []

    def run(cmd, **k):
        ran.append(cmd)
        host = not cmd[0].endswith("nvcc")
        if host and place.host == "missing":
            raise FileNotFoundError(2, "No such file or directory", cmd[0])
        if host and place.host == "fails":
            return subprocess.CompletedProcess(cmd, 1, "", "no Python.h")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    def place():
        del ran[:]
        assert B.build() == B.LIB
        return [os.path.basename(c[c.index("-o") + 1]).split(".tmp")[0] for c in ran]

    place.host = "works"
    monkeypatch.setattr(B.subprocess, "run", run)
    return place


MODULE = os.path.basename(B.PY_LIB)


def test_everything_is_built_once(place):
    assert sorted(place()) == sorted(["a.o", "b.o", MODULE, "libhca.so"])
    assert os.path.exists(B.LIB) and os.path.exists(B.PY_LIB)
    assert place() == []


@pytest.mark.parametrize("host", ["missing", "fails"])
def test_the_library_is_built_without_a_host_compiler_that_works(place, host, capsys):
    place.host = host
    assert sorted(place()) == sorted(["a.o", "b.o", MODULE, "libhca.so"])
    assert os.path.exists(B.LIB) and not os.path.exists(B.PY_LIB)
    assert "was not built" in capsys.readouterr().err
    place.host = "works"
    assert place() == [MODULE] and os.path.exists(B.PY_LIB)


def test_the_library_is_built_without_torch(place, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)   # import torch: ImportError
    assert sorted(place()) == ["a.o", "b.o", "libhca.so"]
    assert os.path.exists(B.LIB) and not os.path.exists(B.PY_LIB)
    assert "was not built" in capsys.readouterr().err


def test_a_kernel_that_does_not_compile_ends_the_build(place, monkeypatch):
    monkeypatch.setattr(B.subprocess, "run", lambda cmd, **k: subprocess.CompletedProcess(cmd, 1, "", "error"))
    with pytest.raises(RuntimeError, match="nvcc failed"):
        B.build()
    assert not os.path.exists(B.LIB)


def test_the_module_is_of_one_python_torch_and_command(place, monkeypatch):
    import sysconfig
    import torch
    assert MODULE == "_hca_py" + sysconfig.get_config_var("EXT_SUFFIX") != "_hca_py.so"
    old = os.path.join(B.HERE, "_hca_py.so")
    place()
    open(old, "w").close()                 # one that any Python would import
    assert place() == [] and not os.path.exists(old)
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "2.0.0")
        assert place() == [MODULE] and place() == []
    assert place() == [MODULE]
    with monkeypatch.context() as m:
        m.setattr(sys, "version", "3.99")
        assert place() == [MODULE]
    place()
    monkeypatch.setenv("CXX", "clang++")
    assert place() == [MODULE] and place() == []


def test_a_module_of_another_torch_is_not_used(monkeypatch):
    import types
    import block_sparse_compressed_gb300 as pkg
    from block_sparse_compressed_gb300 import hca
    import torch
    for version, used in ((torch.__version__, True), ("1.0", False), (None, False)):
        m = types.ModuleType("_hca_py")
        if version:
            m.torch_version = version
        monkeypatch.setitem(sys.modules, pkg.__name__ + "._hca_py", m)
        monkeypatch.setattr(pkg, "_hca_py", m, raising=False)
        assert (hca._extension() is m) == used
