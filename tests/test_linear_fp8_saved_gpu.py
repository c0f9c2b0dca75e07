"""The fp8 layer under hooks that replace what it saves for its backward pass: offloading to the host, copies
laid out otherwise. Gradients are those without hooks, bit for bit; what is no replacement raises."""
import pytest
import torch
import torch.utils.checkpoint

import quantized_zero_communication_gb300 as zpp
from test_fp8_gpu import DEV, gen

pytestmark = pytest.mark.gpu


def case(tokens, n, k):
    g = gen(tokens + n + k)
    x = torch.randn(tokens, k, generator=g, device=DEV).bfloat16().requires_grad_()
    w = torch.randn(n, k, generator=g, device=DEV).requires_grad_()
    return x, w, torch.randn(tokens, n, generator=g, device=DEV).bfloat16()


def shifted(t):
    """The same values one element off every alignment."""
    wide = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    return wide[1:].view(t.shape).copy_(t)


HOOKS = {
    "contiguous": lambda t: t.contiguous().clone(memory_format=torch.contiguous_format),
    "columns": lambda t: t.t().contiguous().t(),
    "shifted": shifted,
    "from the host": lambda t: t.cpu().to(DEV),
}


@pytest.mark.parametrize("tokens,n,k", [(5, 33, 48), (1, 1, 16), (130, 100, 257), (64, 128, 256)])
def test_gradients_under_hooks(tokens, n, k):
    x, w, dy = case(tokens, n, k)
    want = torch.autograd.grad(zpp.linear_fp8(x, w), (x, w), dy)
    held = zpp.quant_fp8(w.detach(), 128, transposed=True)
    for make in HOOKS.values():
        for codes in (None, held):
            with torch.autograd.graph.saved_tensors_hooks(lambda t: t, make):
                y = zpp.linear_fp8(x, w, quantized=codes)
            got = torch.autograd.grad(y, (x, w), dy)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for pin in (False, True):
        with torch.autograd.graph.save_on_cpu(pin_memory=pin):
            y = zpp.linear_fp8(x, w)
        got = torch.autograd.grad(y, (x, w), dy)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_checkpointed_layer():
    x, w, dy = case(21, 50, 72)
    want = torch.autograd.grad(zpp.linear_fp8(x, w), (x, w), dy)
    y = torch.utils.checkpoint.checkpoint(zpp.linear_fp8, x, w, use_reentrant=False)
    got = torch.autograd.grad(y, (x, w), dy)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("make", [lambda t: t.cpu(), lambda t: t[:-1], lambda t: t.to(torch.float16)])
def test_what_is_no_replacement_raises(make):
    x, w, dy = case(20, 40, 64)
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t, make):
        y = zpp.linear_fp8(x, w)
    with pytest.raises(RuntimeError, match="linear_fp8: a saved tensor came back"):
        torch.autograd.grad(y, (x, w), dy)
