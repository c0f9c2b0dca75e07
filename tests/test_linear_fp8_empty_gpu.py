"""The fp8 layer with a weight without rows, its codes made in the call or held by the caller."""
import pytest
import torch

import quantized_zero_communication_gb300 as zpp
from test_fp8_gpu import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", (0, 5))
def test_weight_without_rows(tokens):
    w = torch.zeros(0, 48, device=DEV).requires_grad_()
    x = torch.randn(tokens, 48, device=DEV).bfloat16().requires_grad_()
    for held in (None, zpp.quant_fp8(w.detach(), 128, transposed=True)):
        y = zpp.linear_fp8(x, w, quantized=held)
        assert y.shape == (tokens, 0) and y.dtype == x.dtype
        dx, dw = torch.autograd.grad(y, (x, w), torch.ones_like(y))
        assert dx.shape == x.shape and not dx.any() and dw.shape == w.shape
    with torch.no_grad():
        assert zpp.linear_fp8(x, w, quantized=zpp.quant_fp8(w.detach(), 128)).shape == (tokens, 0)
