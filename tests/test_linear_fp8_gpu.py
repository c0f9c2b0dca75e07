"""The fp8 linear layer: its three products against the same products in 64 bits of the values that its
codes stand for, and its gradient against differences of the quantised layer's own function.

A product's result is within (20 + K / 128) u S + half an ulp of its type (see test_fp8_gpu.py)."""
import gc

import pytest
import torch

import quantized_zero_communication_gb300 as zpp
from test_fp8_gpu import DEV, HALF_ULP, U, gen, spread

pytestmark = pytest.mark.gpu


def value(q, tile):
    return q[0].to(torch.float64) * spread(q[1], tile, *q[0].shape)


def near(got, a, b):
    want, size = a @ b.t(), a.abs() @ b.abs().t()
    tol = (20 + a.shape[1] / 128) * U * size
    half = HALF_ULP[got.dtype]
    tol = tol + half * (want.abs() + tol) + torch.finfo(got.dtype).smallest_normal * half
    assert ((got.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("x_dtype,w_dtype", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32),
                                             (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("shape,n", [((1, 16), 1), ((2, 5, 100), 33), ((130, 257), 129), ((3, 64, 512), 640)])
def test_forward_and_gradients(shape, n, x_dtype, w_dtype):
    g = gen(n)
    x = torch.randn(shape, generator=g, device=DEV).to(x_dtype).requires_grad_()
    w = (0.1 * torch.randn(n, shape[-1], generator=g, device=DEV)).to(w_dtype).requires_grad_()
    y = zpp.linear_fp8(x, w)
    assert y.shape == (*shape[:-1], n) and y.dtype == x_dtype
    dy = torch.randn(y.shape, generator=g, device=DEV).to(x_dtype)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    assert dx.shape == x.shape and dx.dtype == x_dtype and dw.shape == w.shape and dw.dtype == w_dtype
    rows, drows = x.detach().reshape(-1, shape[-1]), dy.reshape(-1, n)
    qw = value(zpp.quant_fp8(w.detach(), 128), 128)
    near(y.detach().reshape(-1, n), value(zpp.quant_fp8(rows), 1), qw)
    near(dx.reshape(-1, shape[-1]), value(zpp.quant_fp8(drows), 1), qw.t())
    near(dw, value(zpp.quant_fp8(drows.t().contiguous()), 1), value(zpp.quant_fp8(rows.t().contiguous()), 1))
    # one gradient alone, codes of the caller, a gradient that is broadcast
    held = zpp.quant_fp8(w.detach(), 128, transposed=True)
    assert torch.equal(zpp.linear_fp8(x, w.detach(), quantized=held), y)
    only, = torch.autograd.grad(zpp.linear_fp8(x, w.detach(), quantized=held), x, dy)
    assert torch.equal(only, dx)
    only, = torch.autograd.grad(zpp.linear_fp8(x.detach(), w), w, dy)
    assert torch.equal(only, dw)
    zpp.linear_fp8(x, w).sum().backward()
    ones, = torch.autograd.grad(zpp.linear_fp8(x, w), x, torch.ones_like(dy))
    assert torch.equal(x.grad, ones)


def test_gradient_is_that_of_differences():
    """With x, w and dy on their codes' grids, and steps that stay on them, the layer's function is the
    plain product: its differences are exact in fp32 and equal the gradient's products."""
    g = gen(1)
    draw = lambda *s: torch.randint(-8, 9, s, generator=g, device=DEV).float()  # noqa: E731
    x, w, dy = draw(40, 128), draw(130, 128), draw(40, 130)
    x[:, 0] = w[:, 0] = 8.0  # every block's scale is the same whatever the others are
    dy[:, 0] = dy[0] = 8.0
    xt, wt = x.bfloat16().requires_grad_(), w.clone().requires_grad_()
    dx, dw = torch.autograd.grad(zpp.linear_fp8(xt, wt), (xt, wt), dy.bfloat16())
    loss = lambda a, b: (zpp.linear_fp8(a.bfloat16(), b).double() * dy.double()).sum()  # noqa: E731
    # (y is bf16: products of a few small integers are exact there, so all but two columns are 0)
    x[:, 2:] = 0
    for i, k in ((0, 1), (17, 1), (39, 1)):
        up, down = x.clone(), x.clone()
        up[i, k], down[i, k] = 1.0, -1.0
        assert loss(up, w) - loss(down, w) == 2 * (dy[i].double() * w[:, k].double()).sum()
        want = (dy[i].double() * w[:, k].double()).sum()
        assert abs(float(dx[i, k]) - want) <= 2.0 ** -8 * abs(want)  # bf16, half a step
    for j, k in ((0, 1), (129, 1)):
        want = (dy[:, j].double() * xt.detach()[:, k].double()).sum()
        assert float(dw[j, k]) == want


def test_layer_without_rows_and_changed_codes():
    w = torch.randn(32, 48, device=DEV).requires_grad_()
    x = torch.zeros(0, 48, dtype=torch.bfloat16, device=DEV).requires_grad_()
    y = zpp.linear_fp8(x, w)
    assert y.shape == (0, 32)
    y.sum().backward()
    assert x.grad.shape == x.shape and (w.grad == 0).all()
    x = torch.randn(5, 48, device=DEV).bfloat16().requires_grad_()
    held = zpp.quant_fp8(w.detach(), 128, transposed=True)
    y = zpp.linear_fp8(x, w, quantized=held)
    zpp.quant_fp8(2 * w.detach(), 128, transposed=True, out=held)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_training_pass_in_a_graph():
    g = gen(3)
    x = torch.randn(64, 256, generator=g, device=DEV).bfloat16().requires_grad_()
    w = torch.randn(96, 256, generator=g, device=DEV).requires_grad_()
    dy = torch.randn(64, 96, generator=g, device=DEV).bfloat16()

    def step():
        y = zpp.linear_fp8(x, w)
        return (y, *torch.autograd.grad(y, (x, w), dy))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [t.clone() for t in step()]
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for k in range(2):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.no_grad():
        dy.mul_(4.0)
    graph.replay()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], 4 * want[1]) and torch.equal(got[2], 4 * want[2])


def test_captured_backward_beside_an_eager_graph_raises():
    g = gen(4)
    x = torch.randn(64, 256, generator=g, device=DEV).bfloat16()
    w = torch.randn(96, 256, generator=g, device=DEV).requires_grad_()
    dy = torch.randn(64, 96, generator=g, device=DEV).bfloat16()
    eager = zpp.linear_fp8(x, w)
    want, = torch.autograd.grad(eager, w, dy, retain_graph=True)

    def capture():
        graph, got = torch.cuda.CUDAGraph(), None
        try:
            with torch.cuda.graph(graph):
                got, = torch.autograd.grad(zpp.linear_fp8(x, w), w, dy)
        except RuntimeError as e:
            return str(e), None
        return graph, got

    said, _ = capture()
    assert isinstance(said, str) and "weight's gradient would go to the default stream" in said
    del eager
    gc.collect()
    graph, got = capture()
    graph.replay()
    assert torch.equal(got, want)


def test_only_gradients_that_are_asked_for():
    g = gen(5)
    x = torch.randn(40, 200, generator=g, device=DEV).bfloat16().requires_grad_()
    w = torch.randn(72, 200, generator=g, device=DEV).requires_grad_()
    y = zpp.linear_fp8(x, w)
    dx, dw = torch.autograd.grad(y, (x, w), torch.ones_like(y), retain_graph=True)
    held = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    one, = torch.autograd.grad(y, x, torch.ones_like(y), retain_graph=True)
    assert torch.equal(one, dx) and torch.cuda.max_memory_allocated() - held < 72 * 200 * 4
    assert torch.equal(torch.autograd.grad(y, w, torch.ones_like(y))[0], dw)


def test_second_derivative_raises():
    x = torch.randn(20, 64, device=DEV).bfloat16().requires_grad_()
    w = torch.randn(48, 64, device=DEV).requires_grad_()
    y = zpp.linear_fp8(x, w)
    dx, = torch.autograd.grad(y.float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiable once"):
        dx.float().sum().backward()
    with torch.no_grad():
        assert not zpp.linear_fp8(x, w).requires_grad
