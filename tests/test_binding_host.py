"""The binding's build: one for every torch, interpreter and source, tried again where it is missing, and never a reason for
the library's build to fail."""
import os
import shutil
import subprocess

import pytest
import torch

import sequence_parallelism_striped_gb300 as sp
from sequence_parallelism_striped_gb300 import build


def test_it_is_there():
    """With a compiler and torch's headers the calls go through the binding."""
    header = os.path.join(os.path.dirname(torch.__file__), "include", "torch", "csrc", "autograd", "python_variable.h")
    if shutil.which("g++") is None or not os.path.exists(header):
        pytest.skip("no compiler or no headers")
    build.build()
    assert os.path.exists(build.binding_path())
    sp.load()
    assert sp._fast is not None


@pytest.mark.gpu
def test_it_is_there_beside_a_gpu():
    test_it_is_there()


def test_another_torch_has_another_binding(monkeypatch):
    here = build.binding_path()
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    assert build.binding_path() != here
    monkeypatch.setattr(sp, "_fast", None)
    sp._bind(sp.library_path())
    assert sp._fast is None  # the one that lies there is not loaded


def test_another_header_has_another_binding(monkeypatch, tmp_path):
    here = build.binding_path()
    monkeypatch.setattr(build, "INCLUDE", str(tmp_path))
    assert build.binding_path() is None
    shutil.copy(os.path.join(build.ROOT, "include", "striped.h"), tmp_path)
    assert build.binding_path() == here
    with open(tmp_path / "striped.h", "a") as f:
        f.write("int another;\n")
    assert build.binding_path() not in (here, None)


def _library(monkeypatch, tmp_path):
    """A build folder with a library that is up to date, and no binding."""
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libstriped.so"))
    (tmp_path / "libstriped.so").write_bytes(b"")


def test_a_missing_binding_is_built_beside_a_library_that_stays(monkeypatch, tmp_path):
    _library(monkeypatch, tmp_path)
    made = []

    def run(cmd, **kw):
        made.append(cmd)
        assert cmd[0] == "g++"  # no source of the library is compiled
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(subprocess, "run", run)
    (tmp_path / "striped_binding.so").write_bytes(b"")  # of another source
    build.build()
    assert len(made) == 1 and sorted(os.listdir(tmp_path)) == sorted(["libstriped.so", os.path.basename(build.binding_path())])
    build.build()
    assert len(made) == 1
    monkeypatch.setattr(torch, "__version__", "9.9.9")  # torch is replaced
    build.build()
    assert len(made) == 2 and os.path.exists(build.binding_path())


@pytest.mark.parametrize("how", ["no compiler", "errors", "another torch's attributes"])
def test_a_failure_leaves_the_library_alone_and_is_tried_again(how, monkeypatch, tmp_path, capsys):
    _library(monkeypatch, tmp_path)
    tries = []

    def run(cmd, **kw):
        tries.append(cmd)
        if how == "no compiler":
            raise FileNotFoundError("g++")
        return subprocess.CompletedProcess(cmd, 1, "", "an error")

    monkeypatch.setattr(subprocess, "run", run)
    if how.startswith("another"):
        monkeypatch.delattr(torch._C, "_GLIBCXX_USE_CXX11_ABI")
    for n in (1, 2):
        assert build.build() == str(tmp_path / "libstriped.so")
        assert "not built" in capsys.readouterr().err
        assert len(tries) == (0 if how.startswith("another") else n)
    assert os.listdir(tmp_path) == ["libstriped.so"]
