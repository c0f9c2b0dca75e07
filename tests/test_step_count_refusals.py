"""Argument checks of the counted AdamW step: every case fails one before any launch (fake
addresses)."""
import math

import pytest
import torch

from quantized_zero_communication_gb300 import binding as zb

INV, MIS, UNS = zb.ZPP_ERR_INVALID_ARG, zb.ZPP_ERR_MISALIGNED, zb.ZPP_ERR_UNSUPPORTED
FAKE = 0x10000
pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="fake-address cases run only where no GPU exists")


def call(num=1, bits=32, g_dt=zb.ZPP_BF16, w_dt=zb.ZPP_BF16, hp=None, scale=0, clip=None, record=FAKE, **f):
    d = dict(n=100, param=FAKE, grad=FAKE, exp_avg=FAKE, exp_avg_sq=FAKE, exp_avg_scale=FAKE,
             exp_avg_sq_scale=FAKE, weight=FAKE)
    d.update(f)
    h = dict(dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=0, seed=0), **(hp or {}))
    if clip is not None:
        clip = zb.AdamwClip(**dict(dict(pre_scale=1.0, max_norm=1.0, workspace=FAKE, out=FAKE), **clip))
    return zb.zpp_adamw_step_counted([zb.AdamwTensor(**d)] * num, g_dt, w_dt, bits, zb.AdamwParams(**h),
                                     scale, clip, record)


def test_what_every_step_checks():
    assert call(num=1025, n=0) == INV and call(n=-1) == INV and call(bits=16) == INV
    for k in ("param", "grad", "exp_avg", "exp_avg_sq"):
        assert call(**{k: 0}) == INV and call(**{k: FAKE + 8}) == MIS
    assert call(bits=8, exp_avg_scale=0) == INV and call(bits=8, exp_avg_scale=FAKE + 2) == MIS
    assert call(w_dt=zb.ZPP_F32) == UNS and call(hp=dict(lr=math.nan)) == INV


def test_record_number_and_clip():
    assert call(record=0) == INV and call(record=FAKE + 8) == MIS
    assert call(hp=dict(step=-1)) == INV and call(scale=FAKE + 2) == MIS
    assert call(scale=FAKE, clip={}) == INV
    for bad in (dict(pre_scale=math.inf), dict(max_norm=0.0), dict(max_norm=-1.0), dict(max_norm=math.nan),
                dict(workspace=0), dict(out=0)):
        assert call(clip=bad) == INV, bad
    assert call(clip=dict(workspace=FAKE + 2)) == MIS and call(clip=dict(out=FAKE + 1)) == MIS
