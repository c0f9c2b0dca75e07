"""What the library's calls answer inside the fp8 layer comes out as ZppError, from the forward and from the
backward pass. The failing calls are stand-ins on the host: they return a status and launch nothing."""
import ctypes

import pytest
import torch

import quantized_zero_communication_gb300 as zpp
from quantized_zero_communication_gb300 import binding as zb
from test_fp8_gpu import DEV, gen

pytestmark = pytest.mark.gpu

CALL = ctypes.CFUNCTYPE(ctypes.c_int, *[ctypes.c_void_p] * 7)


def case():
    g = gen(1)
    x = torch.randn(20, 48, generator=g, device=DEV).bfloat16().requires_grad_()
    return x, torch.randn(33, 48, generator=g, device=DEV).requires_grad_()


def layer(x, w, quant=None, matmul=None):
    address = lambda f, name: ctypes.cast(f, ctypes.c_void_p).value if f else zb._address(name)  # noqa: E731
    return zb._tensors().linear_fp8(address(quant, "zpp_quant_fp8"), address(matmul, "zpp_matmul_fp8"), x, w, None)


def test_forward():
    x, w = case()
    fails = CALL(lambda *args: zb.ZPP_ERR_CUDA)
    for kw, name in ((dict(quant=fails), "zpp_quant_fp8"), (dict(matmul=fails), "zpp_matmul_fp8")):
        with pytest.raises(zpp.ZppError, match=f"{name}: {zpp.zpp_status_string(zb.ZPP_ERR_CUDA)}") as raised:
            layer(x, w, **kw)
        assert raised.value.status == zb.ZPP_ERR_CUDA
    assert torch.equal(layer(x, w), zpp.linear_fp8(x, w))


def test_backward():
    x, w = case()
    real = CALL(zb._address("zpp_matmul_fp8"))
    answers = [0, zb.ZPP_ERR_MISALIGNED]

    def once(*args):
        st = answers.pop(0)
        return st or real(*args)

    held = CALL(once)  # (called again by the backward pass)
    y = layer(x, w, matmul=held)
    with pytest.raises(zpp.ZppError, match="zpp_matmul_fp8") as raised:
        torch.autograd.grad(y, (x, w), torch.ones_like(y))
    assert raised.value.status == zb.ZPP_ERR_MISALIGNED and not answers
    y = zpp.linear_fp8(x, w)
    assert torch.autograd.grad(y, x, torch.ones_like(y))[0].isfinite().all()
