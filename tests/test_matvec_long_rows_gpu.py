"""Rows beyond a cluster's shared memory: code times x is exact, as for shorter rows."""
import pytest
import torch

import quantized_zero_communication_gb300 as zpp

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("bits", [4, 8])
def test_code_times_x_is_exact_in_the_longest_rows(bits):
    """One code and one x per row, so that y is their product times the scale, rounded once: with
    scale = 1 + 2^-23 and the like a second rounding shows."""
    rows, cols, block = 64, 800_003, 128
    n = rows * cols
    g = torch.Generator(device=DEV).manual_seed(1)
    top = 7 if bits == 4 else 127
    at = torch.randint(0, cols, (rows,), generator=g, device=DEV)
    q = torch.randint(-top, top + 1, (rows,), generator=g, device=DEV)
    e = torch.arange(rows, device=DEV) * cols + at
    codes = torch.zeros(n if bits == 8 else (n + 1) // 2, dtype=torch.int64, device=DEV)
    if bits == 8:
        codes[e] = q & 255
    else:
        codes.index_put_((e // 2,), (q & 15) << (4 * (e % 2)), accumulate=True)
    scales = 1 + torch.randint(0, 1 << 23, (-(-n // block),), generator=g, device=DEV).float() * 2.0 ** -23
    x = torch.zeros(1, cols, device=DEV, dtype=torch.float16)
    x[0, at] = (torch.randint(1, 2048, (rows,), generator=g, device=DEV)).half()
    y = zpp.matvec_blockwise(codes.to(torch.uint8), scales, x, rows, block, bits, dtype=torch.float32)
    want = q.double() * x[0, at].double() * scales[e // block].double()
    assert torch.equal(y[0], want.float())
