"""A kernel starts on the current device, whatever device its tensors and its stream belong to. So
calls on tensors of another device make that one current around the library call, and put the old
one back. Without a GPU: the extension and the library are stand-ins that say "device 1" of every
tensor and write down what was current."""
import contextlib
import types

import pytest
import torch

import quantized_zero_communication_gb300 as zpp
from quantized_zero_communication_gb300 import binding as zb

HOME, AWAY = 0, 1
KINDS = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2, torch.uint8: 3, torch.float8_e4m3fn: 4}


@pytest.fixture
def calls(monkeypatch):
    """(name of the library call, device current in it, stream given to it) in their order."""
    seen, current = [], [HOME]

    def enter(ts, table, column, sizes):
        for i, t in enumerate(ts):
            table[8 * i + column] = t.data_ptr()
        return KINDS[ts[0].dtype], AWAY, 1

    def scan(ts, at, counts):
        for i, t in enumerate(ts):
            at[i], counts[i] = t.data_ptr(), t.numel()
        return KINDS[ts[0].dtype], AWAY

    def step(*args):
        if current[0] != args[-1]:
            return False
        seen.append(("zpp_adamw_step_counted", current[0], AWAY))
        return None

    native = types.SimpleNamespace(
        enter=enter, scan=scan, step=step, matvec=lambda *a: None, grad_norm=lambda *a: None,
        probe=lambda t: (t.data_ptr(), t.numel(), KINDS[t.dtype], AWAY, t.is_contiguous()))

    class Library:
        def __getattr__(self, name):
            def call(*args):
                seen.append((name, current[0], args[-1]))
                return zb.ZPP_OK
            return call

    @contextlib.contextmanager
    def device(index):
        before, current[0] = current[0], index
        yield
        current[0] = before
    monkeypatch.setattr(zb, "_tensors", lambda: native)
    monkeypatch.setattr(zb, "lib", lambda: Library())
    monkeypatch.setattr(zb, "_address", lambda name: 1)
    monkeypatch.setattr(zb, "_raw_stream", lambda index: index)
    monkeypatch.setattr(zb, "zpp_grad_norm_workspace", lambda total, count: 8)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    yield seen
    assert current[0] == HOME


def z(n, dtype=torch.float32):
    return torch.zeros(n, dtype=dtype)


def test_gradient_norm(calls):
    zpp.grad_norm([z(10), z(5)], max_norm=1.0)
    assert calls == [("zpp_grad_norm", AWAY, AWAY)]


def test_adamw_step(calls):
    zpp.adamw_step(z(300), z(300), z(300), z(300), step=1, lr=1e-3)
    assert calls == [("zpp_adamw_step", AWAY, AWAY)]


def test_optimiser(calls):
    opt = zpp.AdamW([z(300)])
    opt.step([z(300)])
    opt.step([z(300)])
    assert calls == [("zpp_adamw_step_counted", AWAY, AWAY)] * 2 and opt.steps == 2


def test_product(calls):
    zpp.matvec_blockwise(z(1024, torch.uint8), z(32), z(256, torch.float16), 8, 64, 4)
    assert calls == [("zpp_matvec_blockwise", AWAY, AWAY)]
