"""Muon.step writes parameters, momenta and weights: a graph that kept their old values raises, as after any
write in place, and one that kept nothing of them is not disturbed."""
import pytest
import torch

import quantized_zero_communication_gb300 as zpp
from test_muon_gpu import DEV, matrix

pytestmark = pytest.mark.gpu


def setup():
    params = [torch.randn(40, 70, device=DEV), torch.randn(9, 12, device=DEV)]
    weights = [torch.randn(p.shape, device=DEV).bfloat16() for p in params]
    opt = zpp.Muon(params, weights=weights)
    return params, weights, opt, [matrix(*p.shape, 1) for p in params]


@pytest.mark.parametrize("of", ("params", "weights", "buffers"))
def test_a_graph_of_old_values_raises(of):
    params, weights, opt, grads = setup()
    kept = {"params": params, "weights": weights, "buffers": opt.buffers}[of][1]
    x = torch.randn(3, 12, device=DEV, dtype=kept.dtype).requires_grad_()
    y = torch.nn.functional.linear(x, kept)
    opt.step(grads)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    torch.nn.functional.linear(x, kept).sum().backward()


def test_versions():
    params, weights, opt, grads = setup()
    every = [*params, *weights, *opt.buffers]
    before = [t._version for t in every]
    opt.step(grads, max_norm=1e-3)
    assert all(t._version > v for t, v in zip(every, before))
    assert all(g._version == 0 for g in grads)
    plain = zpp.Muon([params[0]])  # without weights
    plain.step(grads[:1])
    leaf = torch.zeros(40, 70, device=DEV, requires_grad=True)  # a leaf may be stepped
    zpp.Muon([leaf]).step(grads[:1])
    assert leaf.requires_grad and leaf.is_leaf and bool((leaf != 0).any())
    with torch.inference_mode():  # (tensors that count no versions)
        p = torch.zeros(40, 70, device=DEV)
        zpp.Muon([p], weights=[torch.zeros(40, 70, device=DEV).half()]).step(grads[:1])
    assert bool((p != 0).any())
