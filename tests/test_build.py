"""What a build needs and what makes one stale, with stand-ins for the compilers (they make empty
files): the C library without torch, the Python extension for the torch and the Python that load it."""
import os
import subprocess
import sys
import types

import pytest

from quantized_zero_communication_gb300 import build as zbuild


@pytest.fixture
def ran(tmp_path, monkeypatch):
    """Outputs of the commands that a build ran, by file name; those named in `fail` fail."""
    made = types.SimpleNamespace(files=[], fail=())

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        name = os.path.basename(out).split(".tmp")[0]
        if name in made.fail:
            return subprocess.CompletedProcess(cmd, 1, "", "stand-in failure")
        made.files.append(name)
        open(out, "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")
    for name in ("LIB", "EXT", "BUILD"):
        monkeypatch.setattr(zbuild, name, str(tmp_path / os.path.basename(getattr(zbuild, name))))
    if hasattr(zbuild, "EXT_ABI"):
        monkeypatch.setattr(zbuild, "EXT_ABI", str(tmp_path / "_build" / "_tensors.abi"))
    monkeypatch.setattr(zbuild.subprocess, "run", run)
    monkeypatch.setattr(zbuild, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    return made


def test_library_without_torch(ran, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # importing it raises
    assert zbuild.build() == zbuild.LIB and os.path.exists(zbuild.LIB)
    assert "_tensors.so" not in ran.files
    del ran.files[:]
    zbuild.build()
    assert ran.files == []  # and is not stale for want of the extension


def test_library_with_a_torch_without_cuda(ran, monkeypatch):
    torch = types.ModuleType("torch")
    torch.__version__, torch.__file__ = "2.9.0+cpu", "/nowhere/torch/__init__.py"
    torch.version = types.SimpleNamespace(cuda=None)
    torch._C = types.SimpleNamespace(_GLIBCXX_USE_CXX11_ABI=True)
    monkeypatch.setitem(sys.modules, "torch", torch)
    zbuild.build()
    assert os.path.exists(zbuild.LIB) and "_tensors.so" not in ran.files


def test_library_is_there_although_the_extension_fails(ran):
    ran.fail = ("_tensors.so",)
    with pytest.raises(RuntimeError, match="tensor_access.cpp"):
        zbuild.build()
    assert os.path.exists(zbuild.LIB)
