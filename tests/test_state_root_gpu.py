"""The square root behind the 8-bit second-moment states, seen through their block scales.

One Newton step for the root with a fused residual (P. Markstein, Computation of elementary
functions on the IBM RISC System/6000 processor, IBM J. Res. Dev. 34, 1990): with y = 1 / sqrt(v)
within a relative 2^-22.9 (the bound that PTX states for rsqrt.approx.f32) and s = fl(v y), the result
fl(s + (v - s^2) y / 2) lies within 2^-44 of the root before its rounding, where the residual
v - s^2 is exact. So it differs from the correctly rounded root only where the root lies within
2^-44 of the middle of two floats, 2^-24 or more apart: 2 * 2^-44 / 2^-24 = 2^-19 of all values. The
residual has its lowest bit at 2^(e - 46) for v in [2^e, 2^(e+1)), e even or odd, so it is exact
from v = 2^-102 on; below, its rounding (half of 2^-149) is at most 2^-24 of v, 2^-25 of the root, which
with the last rounding keeps the result within one ulp.

The scale is fl(root fl(1/448)): floats one apart give scales at most two apart."""
import numpy as np
import pytest
import torch

import quantized_zero_communication_gb300 as zpp

pytestmark = pytest.mark.gpu

DEV, BLOCK = "cuda:0", 256


def scales_of(values):
    """Block scales of sqrt(v) for v = fl(g g), one g per block (beta2 = 0)."""
    n = len(values) * BLOCK
    g = torch.zeros(len(values), BLOCK, device=DEV)
    g[:, 5] = torch.from_numpy(values).to(DEV)
    p = torch.zeros(n, device=DEV)
    m, v = (torch.zeros(n, device=DEV, dtype=torch.uint8).view(torch.float8_e4m3fn) for _ in range(2))
    a, b = (torch.zeros(len(values), device=DEV) for _ in range(2))
    zpp.adamw_step(p, g.view(-1), m, v, step=1, lr=0.0, betas=(0.9, 0.0), scales=([a], [b]))
    return b.cpu().numpy()


def off(values):
    """Distances in floats from the scale of the correctly rounded root."""
    with np.errstate(under="ignore"):
        root = np.sqrt(values * values)  # fp32, correctly rounded
        want = root * np.float32(1.0 / 448.0)
    return np.abs(scales_of(values).view(np.int32).astype(np.int64) - want.view(np.int32))


def test_root_is_the_rounded_one_but_for_a_few():
    rng = np.random.default_rng(0)
    n = 1 << 19
    exponent = rng.integers(-51, 63, n)
    values = np.ldexp(1 + rng.random(n), exponent).astype(np.float32)
    d = off(values)
    # 2^-19 of 2^19 values are expected to differ, at most: ten is far outside chance
    assert int((d > 0).sum()) <= 10 and int(d.max()) <= 2


def test_root_of_the_smallest_normal_values():
    rng = np.random.default_rng(1)
    n = 1 << 17
    values = np.ldexp(1 + rng.random(n), rng.integers(-63, -51, n)).astype(np.float32)
    with np.errstate(under="ignore"):
        values = values[values * values >= np.float32(2.0 ** -126)]
    assert len(values) > n // 2 and int(off(values).max()) <= 2


def test_root_of_exact_squares():
    values = np.arange(1, 4096, dtype=np.float32)
    assert int(off(values).max()) == 0
