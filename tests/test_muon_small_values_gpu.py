"""Matrices whose squares lie below fp32's range, with an eps below their norm: the norm is that of the definition.

Bounds as in test_muon_gpu.py: the result does not depend on the matrix's scale but for the rounding of the norm
and of the quotient, a few 2^-24, which is within them."""
import pytest
import torch

import quantized_zero_communication_gb300 as zpp
from test_muon_gpu import DEV, USUAL, check_one, exact, gen, matrix, norm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("power", (-60, -75, -80, -90, -100))
@pytest.mark.parametrize("rows,cols", [(60, 200), (300, 130), (5, 3)])
def test_scale_does_not_matter(rows, cols, power):
    x = matrix(rows, cols, rows) * 1e4  # entries about 1
    small = x * 2.0 ** power
    want = zpp.orthogonalize(x, dtype=torch.float16, eps=1e-30)
    assert torch.equal(zpp.orthogonalize(small, dtype=torch.float16, eps=2.0 ** -126), want)
    mixed = [small, x, x * 2.0 ** 40]
    for got in zpp.orthogonalize(mixed, dtype=torch.float16, eps=2.0 ** -126):
        assert torch.equal(got, want)


def test_one_step_of_small_values():
    x = torch.randn(40, 90, generator=gen(1), device=DEV) * 1e-24
    got = zpp.orthogonalize(x, steps=1, eps=1e-30, dtype=torch.float16)
    y = x.double() / norm(x.double())
    check_one(got, y, USUAL)
    # values of very unequal size: the small ones vanish beside the large one
    x[3, 4] = 1.0
    got = zpp.orthogonalize(x, steps=1, eps=1e-30, dtype=torch.float16)
    want = torch.zeros_like(got)
    want[3, 4] = sum(USUAL)
    assert torch.equal(got, want)


def test_norm_beside_eps():
    """Below eps the matrix is divided by eps, whether its squares are in fp32's range or not."""
    x = matrix(50, 80, 2) * 1e4
    for power in (-40, -70, -100):
        small = x * 2.0 ** power
        eps = 8 * norm(small.double())
        want = exact(small, (USUAL,) * 5, eps)
        got = zpp.orthogonalize(small, eps=eps, dtype=torch.float16)
        assert norm(got.double() - want) <= (2.0 ** -11 + 2e-3) * norm(want) + 4000 ** 0.5 * 2.0 ** -25
    assert (zpp.orthogonalize(torch.zeros(7, 9, device=DEV), eps=2.0 ** -126) == 0).all()


def test_muon_step_on_what_a_frozen_matrix_leaves():
    """Momenta that have shrunk for long, beside gradients of zero."""
    p0 = torch.randn(70, 130, generator=gen(3), device=DEV)
    m0 = matrix(70, 130, 4) * 1e4
    results = []
    for scale in (1.0, 2.0 ** -90):
        p = p0.clone()
        opt = zpp.Muon([p], lr=1e-2, eps=2.0 ** -126, buffers=[m0 * scale])
        opt.step([torch.zeros_like(p)])
        results.append(p)
    assert results[1].isfinite().all() and torch.equal(results[0], results[1])
