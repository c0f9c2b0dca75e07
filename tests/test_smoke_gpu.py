"""The smoke check runs where torch's library of solvers cannot be loaded (under a profiler, for one)."""
import pytest
import torch

import __graft_entry__

pytestmark = pytest.mark.gpu


def test_smoke_without_solvers(monkeypatch, capsys):
    def missing(*args, **kwargs):
        raise RuntimeError("Error in dlopen: libtorch_cuda_linalg.so")

    for name in ("svd", "svdvals", "eigh", "eigvalsh", "eig", "eigvals", "qr", "inv", "solve", "cholesky", "lstsq", "lu"):
        monkeypatch.setattr(torch.linalg, name, missing)
    __graft_entry__.smoke()
    assert "Muon step" in capsys.readouterr().out
