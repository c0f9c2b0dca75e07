"""An eps below fp32's normal range: an element without gradient or state has m = 0 over a positive
denominator, so it moves by its decay alone."""
import pytest
import torch

import quantized_zero_communication_gb300 as zpp

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1.1e-38, 1e-40, 1e-45, 1e-60, 1e-300])
def test_zero_gradients_stay_finite(bits, eps):
    n = 1000
    code = torch.float32 if bits == 32 else torch.float8_e4m3fn
    p = torch.ones(n, device=DEV)
    g = torch.zeros(n, device=DEV)
    g[500:] = 1e-3
    m, v = (torch.zeros(n, device=DEV).to(code) for _ in range(2))
    s = [torch.zeros(4, device=DEV) for _ in range(2)]
    zpp.adamw_step(p, g, m, v, step=1, lr=1e-2, eps=eps, weight_decay=0.5,
                   scales=None if bits == 32 else ([s[0]], [s[1]]))
    # decay 1e-2 * 0.5; the others move by lr too: a few roundings of numbers near one
    assert float((p[:500] - (1 - 5e-3)).abs().max()) < 2e-7
    assert float((p[500:] - (1 - 5e-3 - 1e-2)).abs().max()) < 4e-7
