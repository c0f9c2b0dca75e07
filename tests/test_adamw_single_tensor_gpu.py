"""A single tensor in place of a list is that tensor, not the list of its rows: the optimiser takes
what adamw_step and step take."""
import pytest
import torch

import quantized_zero_communication_gb300 as zpp

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("bits", [32, 8])
def test_single_tensor(bits):
    gen = torch.Generator(device=DEV).manual_seed(1)
    p = torch.randn(8, 100, generator=gen, device=DEV)  # rows that are no whole state blocks
    g = torch.randn(8, 100, generator=gen, device=DEV)
    w = torch.zeros(8, 100, device=DEV, dtype=torch.bfloat16)
    q, u = p.clone(), w.clone()
    one, listed = zpp.AdamW(p, state_bits=bits, weights=w, seed=1), zpp.AdamW([q], state_bits=bits, weights=[u], seed=1)
    one.step(g)
    listed.step([g])
    assert torch.equal(p, q) and torch.equal(w, u)
    s = listed.state()
    pick = lambda k: s[k] and [t.clone() for t in s[k]][0]  # noqa: E731
    scales = s["scales"] and tuple(x[0].clone() for x in s["scales"])
    again = zpp.AdamW(p, state_bits=bits, weights=w, seed=1, exp_avg=pick("exp_avg"),
                      exp_avg_sq=pick("exp_avg_sq"), scales=scales, step=s["step"])
    again.step(g)
    listed.step(g)
    assert torch.equal(p, q) and torch.equal(w, u)
