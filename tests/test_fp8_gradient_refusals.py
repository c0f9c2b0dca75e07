"""matmul_fp8 has no derivative: a bias or scales that would need one are refused rather than left without it.
The first test runs without a GPU (the refusal comes before the device is looked at)."""
import pytest
import torch

import quantized_zero_communication_gb300 as zpp


def operands(device, needs):
    e4m3 = torch.float8_e4m3fn
    t = dict(a=torch.zeros(4, 256, device=device).to(e4m3), a_scales=torch.ones(4, 2, device=device),
             b=torch.zeros(200, 256, device=device).to(e4m3), b_scales=torch.ones(2, 2, device=device),
             bias=torch.ones(200, device=device, dtype=torch.bfloat16))
    if needs:
        t[needs].requires_grad_()
    return t


def check(device):
    for needs in ("bias", "a", "a_scales", "b", "b_scales"):
        t = operands(device, needs)
        with pytest.raises(ValueError, match=f"{needs}: .* not differentiable"):
            zpp.matmul_fp8(**t)
        with pytest.raises(ValueError, match=f"{needs}: .* not differentiable"):
            zpp.matmul_fp8(**t, y=torch.zeros(4, 200, device=device, dtype=torch.bfloat16))


def test_operands_that_require_gradients():
    check("cpu")
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA tensors only"):
        zpp.matmul_fp8(**operands("cpu", "bias"))


@pytest.mark.gpu
def test_operands_that_require_gradients_on_the_gpu():
    check("cuda")
    for needs in (None, "bias"):
        t = operands("cuda", needs)
        with torch.no_grad():
            assert (zpp.matmul_fp8(**t) == 1).all()
            y = torch.zeros(4, 200, device="cuda", dtype=torch.bfloat16)
            assert (zpp.matmul_fp8(**t, y=y) == 1).all()
    t = operands("cuda", "bias")
    t["bias"] = t["bias"].detach()
    assert (zpp.matmul_fp8(**t) == 1).all()
    y = zpp.matmul_fp8(**{**t, "bias": None}) + t["bias"].requires_grad_()  # the caller's own addition
    y.sum().backward()
    assert (t["bias"].grad == 4).all()
