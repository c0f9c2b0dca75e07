"""What five Newton-Schulz steps may lose, from the number formats alone: every operand in two fp16, sums
in fp32. A Muon step without momentum, decay or learning-rate adjustment takes parameters of zero to
-lr X in fp32, so the steps' own error is seen beneath the rounding of a 16-bit result.

Roundings, of any direction (s the smaller side, n the longer one; |.| the Frobenius norm). A value in two fp16
is off by half a step of a half step, 2^-22 of itself at most and h = 2^-22 / 3 as a root mean square (uniform,
1 / sqrt(3) each), or by 2^-25 below fp16's normal range (X, held times 2^10: by 2^-35). A product P Q over
K terms with factors off by h, and without the product of their second parts, is off by 3 h |P| |Q| / sqrt(K). So
  A: da = 3 h |X|^2 / sqrt(n) + h |A| + s 2^-25
  B: db = |b| da + 2 |c| da |A| / sqrt(s) + 3 h |c| |A|^2 / sqrt(s) + h |B| + s 2^-25
  X: db |X| / sqrt(s) + 3 h |B| |X| / sqrt(s) + h (|a| |X| + |next X|) + sqrt(s n) 2^-35
The steps after it turn X = U S V^T into U F(S) V^T, F an odd polynomial; an error of any direction they multiply by
the root mean square of F's difference quotients: between two singular values, between one and another's
negative, and between one and 0 for the n - s directions that X lacks.
Cuts, of one direction: a sum's running value is cut to fp32 in each of its K / 16 steps, by 2^-24 of itself in the
mean, half of its end in the mean, so a sum of squares falls short by d(K) = (K / 16) 2^-25 of itself (K up
to a multiple of 64, and 2048 at most: longer sums are added up from such ones by fp32 additions). With t a singular value: A by d(n) t^2, which is d(n) (b t^3 + 2 c t^5) of the next X, A A by d(s) t^4
and B X by d(s) (b t^3 + c t^5); the steps after it multiply that by F'.
All are added up, and 3 times their sum is allowed: roundings are not all independent."""
import math

import pytest
import torch

import quantized_zero_communication_gb300 as zpp
from test_muon_gpu import DEV, HALF, USUAL, exact, matrix, norm, wide

pytestmark = pytest.mark.gpu


def later(t, coefficients):
    """(F(t), F'(t)) of the steps together."""
    v, d = t, torch.ones_like(t)
    for a, b, c in coefficients:
        v, d = v * (a + v * v * (b + v * v * c)), d * (a + v * v * (3 * b + v * v * 5 * c))
    return v, d


def growth(t, n, coefficients):
    """By what the steps multiply an error of any direction beside the singular values t of an X [s, n]."""
    v, d = later(t, coefficients)
    apart = t[:, None] - t
    minus = torch.where(apart.abs() > 1e-9, (v[:, None] - v) / apart, d[:, None])
    plus = (v[:, None] + v) / (t[:, None] + t)
    s = t.numel()
    mean = (minus.square().sum() + plus.square().sum()) / 2 + (n - s) * (v / t).square().sum()
    return float((mean / (s * n)).sqrt())


def lost(x, coefficients, eps=1e-7):
    """(the result in 64 bits, the norm of what the steps may lose)."""
    y = wide(x.double()).cpu()
    y = y / max(norm(y), eps)
    s, n = y.shape
    h, rs = 2.0 ** -22 / 3, s ** 0.5
    cut = lambda k: min(math.ceil(k / 64), 32) * 4 * 2.0 ** -25  # noqa: E731
    low = (s * n) ** 0.5 * 2.0 ** -35
    total = (h * norm(y) + low) * growth(torch.linalg.svdvals(y), n, coefficients)
    for k, (a, b, c) in enumerate(coefficients):
        gram = y @ y.t()
        poly = b * gram + c * gram @ gram
        after = a * y + poly @ y
        x1, a1, b1 = norm(y), norm(gram), norm(poly)
        da = 3 * h * x1 * x1 / n ** 0.5 + h * a1 + s * 2.0 ** -25
        db = abs(b) * da + 2 * abs(c) * da * a1 / rs + 3 * h * abs(c) * a1 * a1 / rs + h * b1 + s * 2.0 ** -25
        dx = db * x1 / rs + 3 * h * b1 * x1 / rs + h * (abs(a) * x1 + norm(after)) + low
        t = torch.linalg.svdvals(y)
        short = cut(n) * (b * t ** 3 + 2 * c * t ** 5).abs() + cut(s) * (abs(c) * t ** 5 + (b * t ** 3 + c * t ** 5).abs())
        d = later(later(t, [(a, b, c)])[0], coefficients[k + 1:])[1]
        total += dx * growth(torch.linalg.svdvals(after), n, coefficients[k + 1:]) + norm(d * short)
        y = after
    return (y if x.shape[0] <= x.shape[1] else y.t()).to(DEV), 3 * total


SHAPES = [(64, 64), (100, 300), (129, 200), (256, 256), (256, 1024), (300, 200), (390, 1000), (513, 512), (1100, 260)]


@pytest.mark.parametrize("kind", ("noise", "strong"))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_five_steps_lose_no_more_than_fp32_sums(rows, cols, kind):
    x = matrix(rows, cols, rows + 5 * cols, kind)
    want, off = lost(x, (USUAL,) * 5)
    assert off < 2.0 ** -12 * norm(want)  # (so that the bound says something)
    p = torch.zeros(rows, cols, device=DEV)
    zpp.Muon([p], lr=1.0, momentum=0.0, weight_decay=0.0, nesterov=False, adjust="none").step([x])
    assert norm(-p.double() - want) <= off
    for dtype in (torch.float16, torch.bfloat16):
        got = zpp.orthogonalize(x, dtype=dtype)
        half = HALF[dtype] * (norm(want) + off) + math.sqrt(want.numel()) * 2.0 ** -25
        assert norm(got.double() - want) <= off + half
    assert zpp.zpp_device_fault() == 0


def test_list_of_several_shapes_and_long_sums():
    xs = [matrix(*s, i, "strong") for i, s in enumerate([(200, 3000), (130, 140), (20, 30), (5000, 160), (700, 300)])]
    ps = [torch.zeros_like(x) for x in xs]
    zpp.Muon(ps, lr=1.0, momentum=0.0, weight_decay=0.0, nesterov=False, adjust="none").step(xs)
    for p, x in zip(ps, xs):
        want, off = lost(x, (USUAL,) * 5)
        assert norm(-p.double() - want) <= off
    again = [torch.zeros_like(x) for x in xs]
    zpp.Muon(again, lr=1.0, momentum=0.0, weight_decay=0.0, nesterov=False, adjust="none").step(xs)
    assert all(torch.equal(p, q) for p, q in zip(ps, again))


def test_result_has_its_types_error():
    """An fp16 result is off by its rounding: half a step of a value just above a power of two is 2^-11 of it, uniform
    roundings are 1 / sqrt(3) of that, and other values have less. What the steps lose vanishes beside it."""
    for rows, cols, kind in ((256, 1024, "noise"), (600, 500, "noise"), (600, 500, "strong")):
        x = matrix(rows, cols, rows, kind).half()
        want = exact(x, (USUAL,) * 5)
        assert norm(zpp.orthogonalize(x).double() - want) <= 3 ** -0.5 * 2.0 ** -11 * norm(want)


@pytest.mark.parametrize("rows,cols", [(4096, 65536), (65536, 4096), (4096, 4096)])
def test_sums_of_any_length(rows, cols):
    """Rows of a Hadamard matrix, all of one singular value, so that the result is the matrix times F(s) / s: what the
    sums' cuts leave shows as a factor. The terms of a sum are one number, so every step of 16 may cut it by nearly a
    whole unit, 2^-23 of the running sum, which is half of its end in the mean: A is short by up to d = 128 * 2^-24 after
    the 128 steps that are made in a row, the next s is a s + b s^3 (1 - d) + c s^5 (1 - d)^2, and B X is short by d as
    well. The fp16 pairs and the fp32 results leave 4 * 2^-22 of each step."""
    n, m = max(rows, cols), min(rows, cols)
    i, j = torch.arange(m, device=DEV)[:, None], torch.arange(n, device=DEV)
    bits = i & j
    for shift in (8, 4, 2, 1):
        bits = bits ^ (bits >> shift)
    x = (1 - 2 * (bits & 1)).half()
    del bits
    x = x if rows <= cols else x.t().contiguous()

    def size(short, each):
        a, b, c = USUAL
        s = m ** -0.5
        for _ in range(5):
            g = s * s * (1 - short)
            s = (a + (b * g + c * g * g) * (1 - short)) * s * (1 + each)
        return s

    want = size(0.0, 0.0)
    d = 128 * 2.0 ** -24
    off = max(abs(size(e * d, f * 4 * 2.0 ** -22) - want) for e in (0, 1) for f in (-1, 1))
    p = torch.zeros(rows, cols, device=DEV)
    zpp.Muon([p], lr=1.0, momentum=0.0, weight_decay=0.0, nesterov=False, adjust="none").step([x])
    got = -p.double() * x.double() * n ** 0.5  # (entries of X are s / sqrt(n))
    assert abs(float(got.mean()) - want) <= off
    assert norm(got - want) <= 2 * off * got.numel() ** 0.5
