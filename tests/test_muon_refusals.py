"""Argument checks of the Newton-Schulz steps and the Muon step: the C ABI's statuses (fake addresses;
every case fails a check before any launch) and the tensor wrappers' messages. Runs without a GPU."""
import array
import math

import pytest
import torch

import quantized_zero_communication_gb300 as zpp
from quantized_zero_communication_gb300 import binding as zb

OK, INV, MIS, UNS = zb.ZPP_OK, zb.ZPP_ERR_INVALID_ARG, zb.ZPP_ERR_MISALIGNED, zb.ZPP_ERR_UNSUPPORTED
FAKE = 0x10000
BF16, F32 = torch.bfloat16, torch.float32
cpu_only = pytest.mark.skipif(torch.cuda.is_available(),
                              reason="fake-address cases run only where no GPU exists")
HELD = array.array("d", [3.4445, -4.7750, 2.0315] * 5)
BROKEN = array.array("d", [3.4445, math.nan, 2.0315])


def steps(held=HELD, num=5, eps=1e-7):
    return zb.NewtonSchulz(held.buffer_info()[0] if held is not None else 0, num, eps)


BAD_STEPS = [steps(None), steps(num=0), steps(num=101), steps(eps=0.0), steps(eps=-1.0),
             steps(eps=math.inf), steps(eps=math.nan), steps(BROKEN, 1)]
BAD_SIZES = [dict(rows=-1), dict(cols=-1), dict(rows=(1 << 30) + 1), dict(cols=(1 << 30) + 1),
             dict(rows=1 << 20, cols=(1 << 18) + 1)]


@cpu_only
def test_orthogonalize_statuses():
    def call(x_dt=zb.ZPP_BF16, out_dt=zb.ZPP_BF16, ns=None, work=FAKE, num=1, **kw):
        d = dict(x=FAKE, out=FAKE, rows=8, cols=16)
        d.update(kw)
        row = zb.Matrix(*(d[k] for k, _ in zb.Matrix._fields_))
        return zb.zpp_orthogonalize([row] * num, x_dt, out_dt, ns or steps(), work)
    assert call(num=0, work=0) == OK and call(rows=0, x=0, out=0, work=0) == OK
    assert call(num=1025, rows=0) == INV
    for bad in BAD_SIZES:
        assert call(**bad) == INV, bad
    for bad in BAD_STEPS:
        assert call(ns=bad) == INV
    assert call(x=0) == INV and call(out=0) == INV and call(work=0) == INV
    assert call(x_dt=3) == INV and call(out_dt=-1) == INV and call(out_dt=zb.ZPP_F32) == UNS
    assert call(x=FAKE + 1) == MIS and call(out=FAKE + 1) == MIS and call(work=FAKE + 64) == MIS
    assert call(x=FAKE + 2, x_dt=zb.ZPP_F32) == MIS
    L = zb.lib()
    assert L.zpp_orthogonalize(None, 1, 1, 1, zb.ctypes.addressof(steps()), FAKE, None) == INV
    assert L.zpp_orthogonalize(FAKE, 0, 1, 1, None, FAKE, None) == INV
    assert L.zpp_orthogonalize_workspace(None, 1) == -1 and L.zpp_orthogonalize_workspace(None, -1) == -1
    size = lambda *s: zb.zpp_orthogonalize_workspace([zb.Matrix(0, 0, *v) for v in s])  # noqa: E731
    assert size() == 0 and size((0, 4)) == 0 and size((-1, 4)) == -1
    # X twice, what it lost, A and B; a list takes no less than its parts
    assert size((64, 128)) >= (3 * 64 * 128 + 2 * 64 * 64) * 2
    assert size(*[(64, 128)] * 3, (7, 9)) >= size((64, 128)) + size((7, 9))


@cpu_only
def test_muon_statuses():
    def call(g_dt=zb.ZPP_BF16, w_dt=zb.ZPP_BF16, work=FAKE, num=1, scale=0, hp=None, **kw):
        d = dict(param=FAKE, grad=FAKE, momentum=FAKE, weight=FAKE, rows=8, cols=16)
        d.update(kw)
        row = zb.MuonTensor(*(d[k] for k, _ in zb.MuonTensor._fields_))
        h = dict(lr=1e-3, momentum=0.95, weight_decay=0.1, nesterov=1, adjust=0, ns=steps())
        h.update(hp or {})
        return zb.zpp_muon_step([row] * num, g_dt, w_dt, zb.MuonParams(*h.values()), scale, work)
    assert call(num=0, work=0) == OK and call(cols=0, param=0, grad=0, momentum=0, work=0) == OK
    assert call(num=1025, rows=0) == INV
    for bad in BAD_SIZES:
        assert call(**bad) == INV, bad
    for bad in BAD_STEPS:
        assert call(hp=dict(ns=bad)) == INV
    for bad in (dict(lr=math.nan), dict(lr=math.inf), dict(weight_decay=math.inf), dict(momentum=1.0),
                dict(momentum=-0.1), dict(momentum=math.nan), dict(nesterov=2), dict(adjust=-1), dict(adjust=3)):
        assert call(hp=bad) == INV, bad
    for k in ("param", "grad", "momentum"):
        assert call(**{k: 0}) == INV
    assert call(work=0) == INV and call(g_dt=3) == INV and call(w_dt=-1) == INV
    assert call(w_dt=zb.ZPP_F32) == UNS
    assert call(param=FAKE + 2) == MIS and call(momentum=FAKE + 2) == MIS and call(grad=FAKE + 1) == MIS
    assert call(weight=FAKE + 1) == MIS and call(scale=FAKE + 2) == MIS and call(work=FAKE + 8) == MIS
    L = zb.lib()
    assert L.zpp_muon_step(None, 0, 1, 1, None, None, FAKE, None) == INV
    assert L.zpp_muon_workspace(None, 1) == -1


def raises(match, fn):
    with pytest.raises(ValueError, match=match):
        fn()


def z(*shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype)


def test_wrapper_checks():
    raises("at least one matrix", lambda: zpp.orthogonalize([]))
    raises("coefficients", lambda: zpp.orthogonalize(z(4, 4), steps=0))
    raises("coefficients", lambda: zpp.orthogonalize(z(4, 4), coefficients=(1.0, 2.0)))
    raises("coefficients", lambda: zpp.orthogonalize(z(4, 4), coefficients=[(1.0, 2.0, 3.0)]))
    raises("x: every tensor needs one dtype", lambda: zpp.orthogonalize([z(4, 4), z(4, 4, dtype=BF16)]))
    raises("CUDA tensors only", lambda: zpp.orthogonalize(z(4, 4)))
    raises("at least one matrix", lambda: zpp.Muon([]))
    raises("at most 1024", lambda: zpp.Muon([z(1, 1)] * 1025))
    raises("adjust", lambda: zpp.Muon([z(4, 4)], adjust="rms"))
    raises("expected a matrix", lambda: zpp.Muon([z(4)]))
    raises("coefficients", lambda: zpp.Muon([z(4, 4)], steps=0))
    raises("CUDA tensors only", lambda: zpp.Muon([z(4, 4)]))
