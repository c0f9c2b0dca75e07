"""Products of more tiles than one round of CTAs takes: pairs of CTAs on 256 x 256 with a scale per row or per
tile, P and Q as they are or exchanged (rows of y off 16 bytes), and the kernels of one CTA with 96 and 128
columns in later rounds. Rings and groups of scales go on from one tile to the next, and a sum of 11 blocks ends
inside a group of 4. Codes are small integers and scales powers of two, so that every sum is exact."""
import pytest
import torch

import quantized_zero_communication_gb300 as zpp
from test_fp8_gpu import DEV, integers, powers, product
from test_linear_fp8_gpu import near, value

pytestmark = pytest.mark.gpu


def check(m, n, k, ta, tb, strides):
    a, b = integers(m, k, m + k), integers(n, k, n + 2 * k)
    sa, sb = powers(m, k, ta, 3), powers(n, k, tb, 4)
    want = product(a, sa, ta, b, sb, tb)[0]
    bias = torch.randint(-9, 9, (n,), device=DEV).float()
    assert torch.equal(zpp.matmul_fp8(a, sa, b, sb, bias=bias, dtype=torch.float32).double(), want + bias.double())
    for first, apart in strides:
        wide = torch.full((m, apart), 7.5, device=DEV)
        zpp.matmul_fp8(a, sa, b, sb, y=wide[:, first:first + n])
        assert torch.equal(wide[:, first:first + n].double(), want)
        assert (wide[:, :first] == 7.5).all() and (wide[:, first + n:] == 7.5).all()
    assert zpp.zpp_device_fault() == 0


@pytest.mark.parametrize("tiles", [(1, 1), (1, 128), (128, 1), (128, 128)])
def test_pairs_in_more_than_one_round(tiles):
    check(2600, 2900, 1290, *tiles, [(0, 2900), (4, 2912), (1, 2903)])


@pytest.mark.parametrize("tiles", [(1, 1), (1, 128), (128, 128)])
@pytest.mark.parametrize("m", (77, 120))
def test_single_ctas_in_more_than_one_round(m, tiles):
    check(m, 40000, 1003, *tiles, [(0, 40000), (3, 40005)])


def test_backward_pass_of_many_tiles():
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(1300, 2600, generator=g, device=DEV).bfloat16().requires_grad_()
    w = (0.1 * torch.randn(2900, 2600, generator=g, device=DEV)).requires_grad_()
    dy = torch.randn(1300, 2900, generator=g, device=DEV).bfloat16()
    y = zpp.linear_fp8(x, w)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    qw = value(zpp.quant_fp8(w.detach(), 128), 128)
    near(y.detach(), value(zpp.quant_fp8(x.detach()), 1), qw)
    near(dx, value(zpp.quant_fp8(dy), 1), qw.t())
    near(dw, value(zpp.quant_fp8(dy.t().contiguous()), 1), value(zpp.quant_fp8(x.detach().t().contiguous()), 1))
