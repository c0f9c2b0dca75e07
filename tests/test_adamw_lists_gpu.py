"""Lists on either side of what a launch's tables take: every tensor of a list is stepped as it is
alone (fp32 states, whose result does not depend on the list), bit for bit."""
import pytest
import torch

import quantized_zero_communication_gb300 as zpp

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("count", [1, 2, 15, 16, 17, 33, 64, 65, 129, 431, 432, 433, 448, 449, 864, 865, 1024])
@pytest.mark.parametrize("length", ["short", "long"])
def test_every_tensor_of_a_list_is_stepped(count, length):
    g = torch.Generator(device=DEV).manual_seed(count)
    sizes = [1 + (i * 37) % 700 + (5000 if length == "long" and i % 3 == 0 else 0) for i in range(count)]
    flat = torch.randn(2, sum(-(-n // 8) * 8 for n in sizes), generator=g, device=DEV)
    at, params, grads = 0, [], []
    for n in sizes:
        params.append(flat[0, at:at + n])
        grads.append(flat[1, at:at + n])
        at += -(-n // 8) * 8
    m, v = ([torch.zeros(n, device=DEV) for n in sizes] for _ in range(2))
    alone = [[t.clone() for t in ts] for ts in (params, grads, m, v)]
    zpp.adamw_step(params, grads, m, v, step=3, lr=1e-2, weight_decay=0.1)
    for p, q, a, b in zip(*alone):
        zpp.adamw_step(p, q, a, b, step=3, lr=1e-2, weight_decay=0.1)
    for got, want in zip((params, m, v), (alone[0], *alone[2:])):
        wrong = [i for i, (x, y) in enumerate(zip(got, want)) if not torch.equal(x, y)]
        assert not wrong, (len(wrong), wrong[:5])
