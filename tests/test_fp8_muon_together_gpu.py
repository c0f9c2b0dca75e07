"""A layer's matrix trained as it would be: fp8 forward and backward passes, a clipped Muon step on the
fp32 master, the rounded weight to codes for the next pass, and one token's answer at the end. Every
step is compared with the definitions in 64 bits, started from the state that the step found."""
import pytest
import torch

import quantized_zero_communication_gb300 as zpp
from test_fp8_gpu import DEV, HALF_ULP, U, gen, grid, spread
from test_muon_gpu import USUAL, exact, norm, rounded

pytestmark = pytest.mark.gpu


def on_grid(x, tile):
    v, scales = grid(x, tile)
    return v * spread(scales, tile, *x.shape)


def near(got, a, b):
    """As in test_fp8_gpu: (20 + K / 128) u S + half an ulp of the output's type."""
    want, size = a @ b.t(), a.abs() @ b.abs().t()
    tol = (20 + a.shape[1] / 128) * U * size
    half = HALF_ULP[got.dtype]
    tol = tol + half * (want.abs() + tol) + torch.finfo(got.dtype).smallest_normal * half
    assert ((got.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("tokens,n,k", [(96, 200, 136), (300, 128, 400)])
def test_layer_trained_in_fp8_by_muon(tokens, n, k):
    g = gen(n)
    master = 0.05 * torch.randn(n, k, generator=g, device=DEV)
    weight = master.bfloat16()
    teacher = torch.randn(n, k, generator=g, device=DEV).bfloat16()
    opt = zpp.Muon([master], lr=1e-2, weight_decay=0.1, adjust="match_rms_adamw", weights=[weight])
    codes = zpp.quant_fp8(weight, 128, transposed=True)
    for _ in range(3):
        x = torch.randn(tokens, k, generator=g, device=DEV).bfloat16()
        w = weight.clone().requires_grad_()
        y = zpp.linear_fp8(x, w, quantized=codes)
        dy = (y.detach().float() - x.float() @ teacher.float().t()).bfloat16()
        dw, = torch.autograd.grad(y, w, dy)
        near(y.detach(), on_grid(x, 1), on_grid(weight, 128))
        near(dw, on_grid(dy.t().contiguous(), 1), on_grid(x.t().contiguous(), 1))

        before, m0 = master.double(), opt.buffers[0].double()
        clip = opt.step([dw], max_norm=1.0)
        c = float(clip[1])
        assert abs(float(clip[0]) - norm(dw.double())) <= 1e-5 * norm(dw.double()) and c < 1.0
        m = 0.95 * m0 + 0.05 * c * dw.double()
        u = 0.05 * c * dw.double() + 0.95 * m
        want = exact(u, (USUAL,) * 5)
        lr = 1e-2 * 0.2 * max(n, k) ** 0.5
        off = lr * (1.5 * norm(rounded(u.float(), (USUAL,) * 5) - want) + 2.0 ** -16 * norm(want))
        want = before * (1 - 1e-2 * 0.1) - lr * want
        assert norm(master.double() - want) <= off + 8 * U * norm(before)
        assert torch.equal(weight, master.bfloat16())

        # the codes of the next pass, into the same buffers
        zpp.quant_fp8(weight, 128, transposed=True, out=codes)
        assert torch.equal(codes[0].to(torch.float64), grid(weight, 128)[0])
        assert torch.equal(codes[2].to(torch.float64), grid(weight.t().contiguous(), 128)[0])
    token = torch.randn(1, k, generator=g, device=DEV).bfloat16()
    near(zpp.matmul_fp8(*zpp.quant_fp8(token), codes[0], codes[1], dtype=torch.float32), on_grid(token, 1),
         on_grid(weight, 128))
    assert zpp.zpp_device_fault() == 0
