"""Python code that runs inside the fp8 layer's call, hooks on what it saves: what it raises comes out as it is.
Checkpoints rely on that: they end a recomputation with an exception of their own."""
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


@pytest.mark.parametrize("early", (True, False))
def test_checkpointed_layers(early):
    x, w, dy = case(16, 64, 64)
    two = lambda t, v: zpp.linear_fp8(zpp.linear_fp8(t, v), v)  # noqa: E731
    want = torch.autograd.grad(two(x, w), (x, w), dy)
    with torch.utils.checkpoint.set_checkpoint_early_stop(early):
        y = torch.utils.checkpoint.checkpoint(two, x, w, use_reentrant=False)
        got = torch.autograd.grad(y, (x, w), dy)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_hooks_exception_comes_out():
    class Mine(Exception):
        pass

    def pack(t):
        raise Mine("no room")

    x, w, dy = case(16, 64, 64)
    with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t):
        with pytest.raises(Mine, match="no room"):
            zpp.linear_fp8(x, w)
    y = zpp.linear_fp8(x, w)  # (nothing is left behind)
    assert torch.autograd.grad(y, x, dy)[0].shape == x.shape
