"""Newton-Schulz steps and the Muon step against their definitions in 64 bits.

One step: with h = 2^-11 (fp16's half step) the operands' roundings leave
  |dX| <= h |X|_2 (|b| |A| + 3 |c| |A|_2 |A| + |B|) + h |B|_2 |X| + 2^-16 |a X|     (Frobenius norms)
(A rounded, its square of rounded factors, B rounded, the fp16 factor X; a X has 20 bits and more),
taken 1.05 times for h^2 and the fp32 sums, and half a step of the output's type.
Several steps multiply what the first ones lose, so no such sum is tight: there the same roundings are
made in 64 bits in torch, and the kernel's error may be 1.5 times that (roundings fall differently
where fp32 sums differ) and the output's, and 2^-16 |X| for the fp32 sums themselves (128 terms and more
of 2^-24 each, multiplied by 3.4^4 at most: 2^-24 * 140 where they add up like noise)."""
import math

import pytest
import torch

import quantized_zero_communication_gb300 as zpp

pytestmark = pytest.mark.gpu

DEV, H = "cuda:0", 2.0 ** -11
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TYPES = (torch.float16, torch.bfloat16, torch.float32)
USUAL = (3.4445, -4.7750, 2.0315)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def norm(x):
    return float(torch.linalg.vector_norm(x))


def wide(x):
    return x if x.shape[0] <= x.shape[1] else x.t()


def exact(x, coefficients, eps=1e-7):
    y = wide(x.double())
    y = y / max(norm(y), eps)
    for a, b, c in coefficients:
        gram = y @ y.t()
        y = a * y + (b * gram + c * gram @ gram) @ y
    return y if x.shape[0] <= x.shape[1] else y.t()


def fp16(x, scale=1.0):
    return (x * scale).half().double() / scale


def rounded(x, coefficients, eps=1e-7):
    """The same with the operands' roundings: X in two fp16, the diagonals of A and B apart, products of
    first parts; of both parts, less the smallest, for a side of at most 128."""
    y = wide(x.double())
    y = y / max(norm(y), eps)
    three = y.shape[0] <= 128
    eye = torch.eye(y.shape[0], dtype=torch.float64, device=DEV)

    def two(v, scale=1.0):
        high = fp16(v, scale)
        return high, fp16(v - high, scale)

    def times(p, q):
        r = p[0] @ q[0]
        return r + p[0] @ q[1] + p[1] @ q[0] if three else r

    for k, (a, b, c) in enumerate(coefficients):
        high, low = two(y, 1024.0)
        y = high + low
        gram = times((high, low), (high.t(), low.t()))
        d = torch.diagonal(gram)
        part = two(gram * (1 - eye))
        off = part[0] + part[1] if three else part[0]
        poly = b * (off + eye * d) + c * ((d[:, None] + d) * off + times(part, part) + eye * d * d)
        e = torch.diagonal(poly)[:, None]
        early = k < len(coefficients) - 3 and not three
        y = a * y + e * (high if early else y) + times(two(poly * (1 - eye)), (high, low))
    return y if x.shape[0] <= x.shape[1] else y.t()


def check_one(got, x, coefficients):
    (a, b, c), y = coefficients, wide(x.double())
    y = y / max(norm(y), 1e-7)
    gram = y @ y.t()
    poly = b * gram + c * gram @ gram
    two = lambda v: float(torch.linalg.matrix_norm(v, 2))  # noqa: E731
    off = H * two(y) * (abs(b) * norm(gram) + 3 * abs(c) * two(gram) * norm(gram) + norm(poly))
    off = 1.05 * (off + H * two(poly) * norm(y)) + 2.0 ** -16 * abs(a) * norm(y)
    want = a * y + poly @ y
    off += HALF[got.dtype] * (norm(want) + off) + math.sqrt(want.numel()) * 2.0 ** -25
    assert norm(wide(got.double()) - want) <= off


def check(got, x, coefficients=(USUAL,) * 5):
    want = exact(x, coefficients)
    off = 1.5 * norm(rounded(x, coefficients) - want) + 2.0 ** -16 * norm(want)
    off += HALF[got.dtype] * (norm(want) + off) + math.sqrt(want.numel()) * 2.0 ** -25
    assert got.shape == x.shape and norm(got.double() - want) <= off
    return off


def matrix(rows, cols, seed, kind="noise"):
    g = gen(seed)
    x = torch.randn(rows, cols, generator=g, device=DEV)
    if kind == "strong":  # a few strong directions
        x += 5 * torch.randn(rows, 3, generator=g, device=DEV) @ torch.randn(3, cols, generator=g, device=DEV)
    if kind == "decades":  # singular values over four decades
        u, s, v = torch.linalg.svd(x.double(), full_matrices=False)
        x = ((u * torch.logspace(0, -4, s.numel(), dtype=torch.float64, device=DEV)) @ v).float()
    return 1e-4 * x


SHAPES = [(1, 1), (1, 7), (5, 1), (8, 8), (33, 70), (70, 33), (64, 65), (128, 128), (129, 257), (300, 200),
          (256, 1024), (1000, 130), (513, 512)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_one_step(rows, cols, dtype):
    x = matrix(rows, cols, rows + cols).to(dtype)
    out = torch.bfloat16 if dtype == torch.float32 else dtype
    for coefficients in (USUAL, (1.5, -0.5, 0.0), (0.0, 1.0, 0.0), (1.0, 0.0, 0.0)):
        got = zpp.orthogonalize(x, steps=1, coefficients=coefficients)
        assert got.dtype == out
        check_one(got, x, coefficients)
    check_one(zpp.orthogonalize(x, 1, dtype=torch.float16), x, USUAL)


@pytest.mark.parametrize("kind", ("noise", "strong", "decades"))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_five_steps(rows, cols, kind):
    x = matrix(rows, cols, rows * 3 + cols, kind)
    check(zpp.orthogonalize(x, dtype=torch.float16), x)
    check(zpp.orthogonalize(x.bfloat16()), x.bfloat16())
    steps = [(3.9, -7.0, 3.2), (3.4, -4.8, 2.0), (2.0, -1.5, 0.5)]
    check(zpp.orthogonalize(x, 3, steps, dtype=torch.float16), x, steps)
    assert zpp.zpp_device_fault() == 0


def test_large_matrices():
    for rows, cols in ((1024, 2500), (2176, 1024), (1500, 1500)):
        x = matrix(rows, cols, rows, "strong")
        got = zpp.orthogonalize(x, dtype=torch.float16)
        check(got, x)
        again = zpp.orthogonalize(x, dtype=torch.float16)
        assert torch.equal(got, again)


@pytest.mark.parametrize("rows,cols", [(100, 6000), (9000, 40), (300, 20000), (7000, 200), (1, 40000), (700, 9000)])
def test_long_matrices(rows, cols):
    """Few tiles of long sums: shared between CTAs and joined."""
    x = matrix(rows, cols, rows, "strong")
    got = zpp.orthogonalize(x, dtype=torch.float16)
    check(got, x)
    assert torch.equal(got, zpp.orthogonalize(x, dtype=torch.float16))
    check_one(zpp.orthogonalize(x, 1, dtype=torch.float16), x, USUAL)
    short = [matrix(20, 30, i) for i in range(3)]  # beside short ones
    for y, z in zip(zpp.orthogonalize([short[0], x, *short[1:]], dtype=torch.float16), (short[0], x, *short[1:])):
        check(y, z)
    assert zpp.zpp_device_fault() == 0


def test_lists_of_many_shapes_and_places():
    """More shapes and matrices than one batch holds; views that start anywhere."""
    shapes = [(1 + i % 23, 3 + i % 19) for i in range(300)]
    flat = matrix(1, sum(r * c for r, c in shapes) + 1, 5).reshape(-1).half()
    for start in (0, 1):
        xs, at = [], start
        for r, c in shapes:
            xs.append(flat[at:at + r * c].view(r, c))
            at += r * c
        got = zpp.orthogonalize(xs)
        for x, y in zip(xs[::17], got[::17]):
            check(y, x)
        alone = [zpp.orthogonalize(x) for x in xs[:40]]
        assert all(torch.equal(a, b) for a, b in zip(alone, got))
        copies = [x.clone() for x in xs]
        same = zpp.orthogonalize(copies, out=copies)  # in place
        assert all(a is b and torch.equal(a, c) for a, b, c in zip(same, copies, got))
    assert zpp.orthogonalize([xs[0].new_zeros(0, 5), xs[0]])[0].shape == (0, 5)


def test_special_matrices():
    assert (zpp.orthogonalize(torch.zeros(40, 50, device=DEV)) == 0).all()
    x = matrix(60, 200, 9)
    x[30:] = 0  # rows without a value stay so, and columns
    x[:, 7] = 0
    got = zpp.orthogonalize(x)
    assert (got[30:] == 0).all() and (got[:, 7] == 0).all()
    check(got, x)
    one = torch.zeros(33, 44, device=DEV)
    one[3, 5] = -2e-3  # a single value: the steps of the number 1
    got = zpp.orthogonalize(one, dtype=torch.float16)
    check(got, one)
    for scale in (1e-3, 1e10):  # the result does not depend on the scale
        check(zpp.orthogonalize(x * scale, dtype=torch.float16), x * scale)
    tiny = x * 1e-9  # far below eps: divided by eps
    want = exact(tiny, (USUAL,) * 5)
    assert norm(zpp.orthogonalize(tiny, dtype=torch.float16).double() - want) <= 1e-2 * norm(want) + 60 * 200 * 2.0 ** -25
    for bad in (float("nan"), float("inf"), 1e30):
        y = x.clone()
        y[2, 3] = bad
        assert zpp.orthogonalize(y).isnan().all()
    # two matrices of one call do not touch each other
    got = zpp.orthogonalize([y, x])
    assert got[0].isnan().all() and torch.equal(got[1], zpp.orthogonalize(x))


def muon_reference(p, g, m, c, opt, lr):
    p, g, m = p.double(), g.double() * c, m.double()
    m = opt.momentum * m + (1 - opt.momentum) * g
    u = (1 - opt.momentum) * g + opt.momentum * m if opt.nesterov else m
    rows, cols = p.shape
    adj = {"original": math.sqrt(max(1.0, rows / cols)), "match_rms_adamw": 0.2 * math.sqrt(max(rows, cols)),
           "none": 1.0}[opt.adjust]
    want = exact(u, (USUAL,) * 5)
    off = 1.5 * norm(rounded(u.float(), (USUAL,) * 5) - want) + 2.0 ** -16 * norm(want)
    return p * (1 - lr * opt.weight_decay) - lr * adj * want, m, lr * adj * off


@pytest.mark.parametrize("g_dtype,w_dtype", [(torch.float32, None), (torch.bfloat16, torch.bfloat16),
                                             (torch.float16, torch.float16)])
@pytest.mark.parametrize("adjust,nesterov", [("original", True), ("match_rms_adamw", False), ("none", True)])
def test_muon_steps(adjust, nesterov, g_dtype, w_dtype):
    shapes = [(64, 128), (130, 33), (64, 128), (7, 9), (257, 64)]
    params = [0.02 * torch.randn(s, generator=gen(i), device=DEV) for i, s in enumerate(shapes)]
    weights = None if w_dtype is None else [torch.empty(s, dtype=w_dtype, device=DEV) for s in shapes]
    opt = zpp.Muon(params, lr=1e-2, adjust=adjust, nesterov=nesterov, weights=weights)
    for t in range(3):
        grads = [matrix(*s, 10 * t + i, "strong").to(g_dtype) for i, s in enumerate(shapes)]
        lr = 1e-2 / (t + 1)
        before = [(p.clone(), m.clone()) for p, m in zip(params, opt.buffers)]
        got = opt.step(grads, lr=lr, max_norm=None if t == 0 else 1e-3, pre_scale=0.5 if t == 2 else None)
        c = 1.0 if t == 0 else float(got[1])
        assert (got is None) == (t == 0)
        for i, ((p0, m0), g) in enumerate(zip(before, grads)):
            p, m, off = muon_reference(p0, g, m0, c, opt, lr)
            assert ((opt.buffers[i].double() - m).abs()
                    <= 4 * 2.0 ** -24 * (m0.abs() + g.double().abs() * c) + 1e-40).all()
            assert norm(params[i].double() - p) <= off + 4 * 2.0 ** -24 * (norm(p) + norm(p0))
            if weights is not None:
                assert torch.equal(weights[i], params[i].to(w_dtype))


def test_muon_skips_what_is_not_finite_and_resumes():
    params = [torch.randn(40, 70, generator=gen(1), device=DEV)]
    weights = [torch.zeros(40, 70, dtype=torch.bfloat16, device=DEV)]
    opt = zpp.Muon(params, weights=weights)
    g = matrix(40, 70, 2)
    opt.step(g)
    kept = [t.clone() for t in (params[0], opt.buffers[0], weights[0])]
    bad = g.clone()
    bad[1, 1] = float("inf")
    got = opt.step(bad, max_norm=1.0)
    assert got[0].isinf() or got[0].isnan()
    opt.step(g, grad_scale=torch.full((1,), float("nan"), device=DEV))
    assert all(torch.equal(a, b) for a, b in zip(kept, (params[0], opt.buffers[0], weights[0])))
    other = zpp.Muon([params[0].clone()], **{k: [t.clone() for t in v] for k, v in opt.state().items()})
    opt.step(g, grad_scale=torch.full((1,), 0.5, device=DEV))
    other.step([0.5 * g])
    assert torch.equal(other.params[0], params[0]) and torch.equal(other.buffers[0], opt.buffers[0])


def test_muon_of_views_that_start_anywhere():
    """Stacks of odd-sized matrices: parameters, gradients, momenta and weights off every alignment."""
    shapes = (3, 37, 53)
    stack = torch.randn(shapes, generator=gen(1), device=DEV)
    apart = [t.clone() for t in stack]
    low = torch.zeros(shapes, dtype=torch.bfloat16, device=DEV)
    g = torch.stack([matrix(37, 53, i) for i in range(3)]).bfloat16()
    opt = zpp.Muon(list(stack), weights=list(low), buffers=list(torch.zeros(shapes, device=DEV)))
    plain = zpp.Muon(apart)
    for _ in range(2):
        a = opt.step(list(g), max_norm=1e-3)
        b = plain.step([t.clone() for t in g], max_norm=1e-3)
        assert torch.equal(a, b)
    assert torch.equal(stack, torch.stack(apart)) and torch.equal(low, stack.bfloat16())


def test_muon_in_a_graph_and_beside_another_stream():
    params = [torch.randn(s, generator=gen(1), device=DEV) for s in ((96, 64), (64, 200))]
    twin = [p.clone() for p in params]
    opt, plain = zpp.Muon(params, lr=1e-2), zpp.Muon(twin, lr=1e-2)
    g = [matrix(*p.shape, 3) for p in params]
    opt.step(g, max_norm=1e-3)
    plain.step(g, max_norm=1e-3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step(g, max_norm=1e-3)
    for _ in range(3):
        graph.replay()
        plain.step(g, max_norm=1e-3)
    assert all(torch.equal(a, b) for a, b in zip(params, twin))
    # two lists on two streams at once
    xs = [matrix(200, 300, i).bfloat16() for i in range(8)]
    want = [zpp.orthogonalize(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i, x in enumerate(xs):
        with torch.cuda.stream(streams[i % 2]):
            got.append(zpp.orthogonalize(x))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
