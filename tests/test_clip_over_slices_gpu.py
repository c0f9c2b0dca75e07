"""The clip factor of a gradient whose slices lie in several optimisers, as ranks hold them: each
takes its own norm, their squares are added (by an all-reduce between ranks), and every one steps by the
factor of the whole."""
import math

import pytest
import torch

import quantized_zero_communication_gb300 as zpp

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def factor_of(norms, max_norm):
    total = torch.stack(norms).square().sum().sqrt()
    return torch.where(total.isfinite(), (max_norm / total).clamp(max=1.0), math.nan).reshape(1)


@pytest.mark.parametrize("bad", [False, True])
def test_slices_step_as_the_whole(bad):
    n, parts = 40_000, 4
    gen = torch.Generator(device=DEV).manual_seed(1)
    grad = torch.randn(n, generator=gen, device=DEV)
    if bad:
        grad[12_345] = math.inf  # one slice overflows: no slice steps
    whole = torch.ones(n, device=DEV)
    flat = whole.clone()
    opt = zpp.AdamW([whole], lr=1e-2)
    opts = [zpp.AdamW([s], lr=1e-2) for s in flat.chunk(parts)]
    for _ in range(2):
        opt.step([grad], max_norm=1.0)
        norms = [zpp.grad_norm([g])[0] for g in grad.chunk(parts)]
        factor = factor_of(norms, 1.0)
        for o, g in zip(opts, grad.chunk(parts)):
            o.step([g], grad_scale=factor)
    # the factor differs by the norm's roundings (1e-5 at most), m and sqrt(v) by as much, and the
    # update, their quotient, by twice that: 2 steps of 1e-2
    assert float((whole - flat).abs().max()) < 2 * 1e-2 * 4e-5
    assert [o.steps for o in opts] == [opt.steps] * parts == [0 if bad else 2] * parts
    assert bool((flat == 1).all()) == bad
