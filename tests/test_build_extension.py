"""The Python extension belongs to the torch and the Python that it was compiled against: with
another one it is compiled again, and not loaded before."""
import os
import sys
import types

import pytest
from test_build import ran  # noqa: F401 (the stand-in compilers)

from quantized_zero_communication_gb300 import binding as zb
from quantized_zero_communication_gb300 import build as zbuild


def test_another_torch_or_python_makes_it_stale(ran, monkeypatch):  # noqa: F811
    import torch
    zbuild.build()
    assert "_tensors.so" in ran.files
    del ran.files[:]
    zbuild.build()
    assert ran.files == []
    monkeypatch.setattr(torch, "__version__", "99.0+cu130")
    zbuild.build()
    assert ran.files == ["_tensors.so"]  # the library does not depend on it
    config = zbuild.sysconfig.get_config_var
    monkeypatch.setattr(zbuild.sysconfig, "get_config_var",
                        lambda name: "cpython-399-other" if name == "SOABI" else config(name))
    del ran.files[:]
    zbuild.build()
    assert ran.files == ["_tensors.so"]


def test_one_of_another_torch_is_not_loaded(ran, monkeypatch):  # noqa: F811
    import torch
    zbuild.build()
    monkeypatch.setattr(zb, "_tensors_module", None)
    monkeypatch.setattr(torch, "__version__", "99.0+cu130")
    loaded = types.ModuleType("stand-in")
    package = "quantized_zero_communication_gb300"
    monkeypatch.setitem(sys.modules, package + "._tensors", loaded)
    monkeypatch.setattr(sys.modules[package], "_tensors", loaded, raising=False)
    with pytest.raises(RuntimeError, match="99.0"):
        zb._tensors()
    assert os.path.exists(zbuild.EXT)
