"""The AdamW step and the gradient norm against their definitions in 64 bits.

Tolerances, with u = 2^-24 (half an ulp of fp32, relative) and square root and division
allowed two ulps (4u) each:
  m  two products (factor and product rounded: 2u; the gradient's scale one more) and a sum:
     |dm| <= 4u (|b1 m| + |(1-b1) g|)
  v  |dv| <= 6u v;  sqrt(v): 3u + 4u = 7u
  p  the quotient: 7u + 3u for the denominator, 4u the division, 2u step size and product,
     and m's own error; the two final sums 3u of their terms:
     |dp| <= u |p'| + 3u (|decay p| + |step|) + 16u |step| + |step size| dm / denominator
All are doubled for second-order terms."""
import math

import pytest
import torch

import quantized_zero_communication_gb300 as zpp
from quantized_zero_communication_gb300 import binding as zb

pytestmark = pytest.mark.gpu

DEV, U, BLOCK = "cuda:0", 2.0 ** -24, 256
HP = dict(lr=3e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1)
SIZES = (1, 7, 255, 256, 257, 2047, 2048, 2049, 5000, 70_001)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(n, sigma, g):
    return torch.randn(n, generator=g, device=DEV) * sigma


def bits_of(i, seed, step):
    """The header's hash of element numbers i, in Python integers mod 2^32 (as int64)."""
    M = 0xFFFFFFFF
    key = ((seed * 0x9E3779B9) ^ (step * 0x510E527F)) & M
    x = ((i & M) * 0x9E3779B9 + (i >> 32) * 0xA54FF53B + key) & M
    x = ((x ^ (x >> 16)) * 0xBB67AE85 + key) & M
    x = ((x ^ (x >> 15)) * 0x9B05688D) & M
    return x ^ (x >> 16)


def reference(p, g, m, v, step, c=1.0):
    """(p, m, v, tolerances) in fp64 after one step."""
    b1, b2 = HP["betas"]
    p, g, m, v = (t.double() for t in (p, g, m, v))
    g = g * c
    dm = 8 * U * ((b1 * m).abs() + ((1 - b1) * g).abs())
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    size = HP["lr"] / (1 - b1 ** step)
    den = v.sqrt() / math.sqrt(1 - b2 ** step) + HP["eps"]
    upd, dec = size * m / den, HP["lr"] * HP["weight_decay"] * p
    new = p - dec - upd
    dp = 2 * U * (new.abs() + 3 * (dec.abs() + upd.abs()) + 16 * upd.abs()) + size * dm / den
    return new, m, v, dp, dm, 12 * U * v


def within(got, want, tol, what):
    # the last term: results below fp32's normal range round absolutely
    bad = (got.double() - want).abs() > tol + 2.0 ** -148
    assert not bool(bad.any()), (what, int(bad.sum()), (got.double() - want).abs().max())


def rounded(p, dtype):
    return p.to(dtype)


def decode(codes, scale):
    n = codes.numel()
    return codes.double() * scale.double().repeat_interleave(BLOCK)[:n]


@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("weight", [None, torch.bfloat16, torch.float16])
def test_fp32_states(grad, weight):
    g_ = gen(1)
    P = [normal(n, 0.02, g_) for n in SIZES]
    G = [normal(n, 1e-3, g_).to(grad) for n in SIZES]
    M = [normal(n, 1e-3, g_) for n in SIZES]
    V = [normal(n, 1e-3, g_).square() for n in SIZES]
    W = None if weight is None else [torch.full((n,), 7.0, device=DEV, dtype=weight) for n in SIZES]
    want = [reference(p, g, m, v, 11) for p, g, m, v in zip(P, G, M, V)]
    zpp.adamw_step(P, G, M, V, step=11, weights=W, **HP)
    for i, (p, m, v, dp, dm, dv) in enumerate(want):
        within(P[i], p, dp, "p")
        within(M[i], m, dm, "m")
        within(V[i], v, dv, "v")
        if W is not None:
            assert torch.equal(W[i], rounded(P[i], weight))


@pytest.mark.parametrize("offset", [0, 16, 32])
@pytest.mark.parametrize("bits", [32, 8])
def test_alignment_and_bounds(offset, bits):
    """Buffers that start 16-, 32- or 64-byte aligned (in their own elements), with guard
    elements on both sides that must stay."""
    n, g_ = 5003, gen(2)

    def at(dtype, count=n, fill=None):
        item = dtype.itemsize
        pad = offset // item if offset else 0
        buf = torch.full(((count + pad) * item + 256,), 0x5A, dtype=torch.uint8, device=DEV)
        t = buf[pad * item:(pad + count) * item].view(dtype)
        if fill is not None:
            t.copy_(fill)
        return buf, t, pad * item, (pad + count) * item

    code = torch.float32 if bits == 32 else torch.float8_e4m3fn
    parts = [at(torch.float32, fill=normal(n, 0.02, g_)),
             at(torch.bfloat16, fill=normal(n, 1e-3, g_).bfloat16()),
             at(code, fill=torch.zeros(n, device=DEV).to(code)),
             at(code, fill=torch.zeros(n, device=DEV).to(code)), at(torch.bfloat16)]
    blocks = -(-n // BLOCK)
    scales = [at(torch.float32, blocks, torch.zeros(blocks, device=DEV)) for _ in range(2)]
    p, g, m, v, w = (x[1] for x in parts)
    plain = [t.clone() for t in (p, g, m, v, w)] + [x[1].clone() for x in scales]
    sc = lambda a, b: None if bits == 32 else ([a], [b])  # noqa: E731
    zpp.adamw_step(p, g, m, v, step=1, weights=[w], scales=sc(scales[0][1], scales[1][1]), **HP)
    zpp.adamw_step(*plain[:4], step=1, weights=[plain[4]], scales=sc(*plain[5:]), **HP)
    for got, want in zip([p, g, m, v, w] + [x[1] for x in scales], plain):
        assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
    for buf, _, lo, hi in parts + (scales if bits == 8 else []):
        assert bool((buf[:lo] == 0x5A).all()) and bool((buf[hi:] == 0x5A).all())


def check_fp8(P, G, M, V, ms, vs, step, seed, c=1.0):
    """Runs one 8-bit step on lists and checks every output against the definition."""
    n_before, want = 0, []
    for p, g, m, v, a, b in zip(P, G, M, V, ms, vs):
        new = reference(p, g, decode(m, a), decode(v, b) ** 2, step, c)
        i = torch.arange(p.numel(), device=DEV) + n_before
        n_before += -(-p.numel() // BLOCK) * BLOCK
        want.append((new, bits_of(i, seed, step)))
    scale = None if c == 1.0 else torch.tensor([c], device=DEV)
    zpp.adamw_step(P, G, M, V, step=step, scales=(ms, vs), seed=seed, grad_scale=scale, **HP)
    for k, ((p, m, v, dp, dm, dv), bits) in enumerate(want):
        within(P[k], p, dp, "p")
        n, r = p.numel(), v.sqrt()
        pad = -n % BLOCK
        for codes, scale, x, tol, draw, keep in ((M[k], ms[k], m, dm, bits & 65535, False),
                                                (V[k], vs[k], r, 16 * U * r, bits >> 16, True)):
            blocks = torch.nn.functional.pad(x, (0, pad)).view(-1, BLOCK)
            amax = blocks.abs().amax(1)
            slack = torch.nn.functional.pad(tol, (0, pad)).view(-1, BLOCK).amax(1)
            within(scale, amax / 448, slack / 448 + 2 * U * amax / 448, "scale")
            s = scale.double().repeat_interleave(BLOCK)[:n]
            live = s > 0
            assert bool((codes.float()[~live] == 0).all())
            y = torch.where(live, x / s.clamp(min=1e-300), torch.zeros_like(x))
            h = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
            at = y.abs() / h + (draw.double() + 0.5) / 65536
            low = torch.floor(at)
            q = (low * h).clamp(max=448.0)
            if keep:
                q = torch.where(y > 0, q.clamp(min=2.0 ** -9), q)
            got = codes.double()
            # fp32 puts x / scale within its own error of the exact one: where that reaches the
            # next grid point, either neighbour is right
            near = (tol + 6 * U * x.abs()) / s.clamp(min=1e-300) / h + 2.0 ** -18
            edge = ((at - low) < near) | ((at - low) > 1 - near)
            same = got.abs() == q
            beside = (got.abs() - q).abs() <= 2 * h  # 2h: across a power of two
            assert bool((same | (edge & beside)).all()), (k, int((~same).sum()))
            assert int((~same).sum()) < 1e-3 * n + 3
            assert bool((torch.sign(got) * torch.sign(x) >= 0).all())


@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16, torch.float16])
def test_fp8_states(grad):
    """Two steps from zero states, then one with a gradient scale: lists of odd sizes, so
    element numbers count blocks through the tensors."""
    g_ = gen(3)
    P = [normal(n, 0.02, g_) for n in SIZES]
    M, V = ([torch.zeros(n, device=DEV).to(torch.float8_e4m3fn) for n in SIZES] for _ in range(2))
    ms, vs = ([torch.zeros(-(-n // BLOCK), device=DEV) for n in SIZES] for _ in range(2))
    for step, c in ((1, 1.0), (2, 1.0), (3, 0.37)):
        # magnitudes over five decades inside a block, zeros among them
        G = [(normal(n, 1e-3, g_) * torch.exp(-3 * torch.rand(n, generator=g_, device=DEV) ** 2 * 4)
              * (torch.rand(n, generator=g_, device=DEV) > 0.1)).to(grad) for n in SIZES]
        check_fp8(P, G, M, V, ms, vs, step, seed=0xFEDCBA98, c=float(torch.tensor(c)))


def test_fp8_zero_gradients_and_tiny_blocks():
    """An all-zero block holds scale 0 and codes 0 and moves nothing but the decay; a block
    of fp32's smallest gradients neither divides by zero nor overflows."""
    n = 3 * BLOCK
    g = torch.zeros(n, device=DEV)
    g[BLOCK:2 * BLOCK] = 1e-30
    g[2 * BLOCK:] = 1e-37
    p = torch.ones(n, device=DEV)
    m, v = (torch.zeros(n, device=DEV).to(torch.float8_e4m3fn) for _ in range(2))
    a, b = (torch.zeros(3, device=DEV) for _ in range(2))
    zpp.adamw_step(p, g, m, v, step=1, scales=([a], [b]), **HP)
    assert float(a[0]) == 0 and float(b[0]) == 0
    assert bool((m[:BLOCK].float() == 0).all()) and bool((v[:BLOCK].float() == 0).all())
    for t in (p, m.float(), v.float(), a, b):
        assert bool(torch.isfinite(t).all())
    decayed = 1 - HP["lr"] * HP["weight_decay"]
    assert abs(float(p[0]) - decayed) < 2e-7


def test_fp8_running_average_moves():
    """Stochastic rounding: v follows its average although each step moves it by a
    thousandth, far below the codes' spacing (an eighth to a sixteenth): 400 steps take v to
    0.999^400 v0 + (1 - 0.999^400) g^2 within the noise of 2^18 elements. Rounding to nearest
    would leave v where it was (ratio 1)."""
    n = 1 << 18
    p = torch.zeros(n, device=DEV)
    g = torch.full((n,), 1e-3, device=DEV)
    opt = zpp.AdamW([p], lr=0.0, weight_decay=0.0, state_bits=8, seed=5,
                    exp_avg=[torch.full((n,), 448.0, device=DEV).to(torch.float8_e4m3fn)],
                    # values from 300 to 448, so the block's largest does not fix them all
                    exp_avg_sq=[(300 + 148 * torch.rand(n, generator=gen(4), device=DEV)
                                 ).to(torch.float8_e4m3fn)],
                    scales=([torch.full((n // BLOCK,), 1e-3 / 448, device=DEV)],
                            [torch.full((n // BLOCK,), 1e-2 / 448, device=DEV)]))
    v0 = decode(opt.exp_avg_sq[0], opt.scales[1][0]).square()
    for _ in range(400):
        opt.step([g])
    v = decode(opt.exp_avg_sq[0], opt.scales[1][0]).square()
    keep = 0.999 ** 400
    want = keep * v0 + (1 - keep) * 1e-6
    # A step moves r by 0.0005 r, so it rounds away from its neighbour with probability p <=
    # 0.0005 r / h <= 0.008 and adds at most p h^2 to r's variance: after 400 steps at most 3.2
    # h^2 <= 3.2 (r / 8)^2 = 0.05 r^2, which is by how much the mean of r^2 may exceed the square
    # of the (unbiased) mean. The 2^18 elements' own noise is below 0.001.
    ratio = float(v.mean() / want.mean())
    assert 0.98 < ratio < 1.08, ratio


@pytest.mark.parametrize("bits", [32, 8])
def test_infinite_and_nan_gradients_stay_in_their_element(bits):
    n, g_ = 4 * BLOCK, gen(5)
    bad = torch.tensor([3, 300, 301, 1023], device=DEV)
    g = normal(n, 1e-3, g_)
    g[bad] = 0
    code = torch.float32 if bits == 32 else torch.float8_e4m3fn
    out = []
    for poison in (False, True):
        x = g.clone()
        if poison:
            x[bad] = torch.tensor([math.inf, -math.inf, math.nan, math.inf], device=DEV)
        p = torch.ones(n, device=DEV)
        m, v = (torch.zeros(n, device=DEV).to(code) for _ in range(2))
        a, b = (torch.zeros(4, device=DEV) for _ in range(2))
        zpp.adamw_step(p, x, m, v, step=1, scales=None if bits == 32 else ([a], [b]), **HP)
        out.append((p, m.float(), v.float(), a, b))
    clean, hurt = out
    rest = torch.ones(n, dtype=torch.bool, device=DEV)
    rest[bad] = False
    for k in range(3):
        assert torch.equal(clean[k][rest], hurt[k][rest])
    for k in (3, 4):
        assert torch.equal(clean[k], hurt[k])
    assert not bool(torch.isfinite(hurt[1][bad]).any()) and not bool(torch.isfinite(hurt[2][bad]).any())


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("c", [math.nan, math.inf])
def test_non_finite_scale_skips_the_step(bits, c):
    n, g_ = 3001, gen(6)
    code = torch.float32 if bits == 32 else torch.float8_e4m3fn
    ts = [normal(n, 1.0, g_), normal(n, 1.0, g_), normal(n, 1.0, g_).to(code),
          normal(n, 1.0, g_).abs().to(code)]
    sc = [torch.ones(12, device=DEV) for _ in range(2)]
    w = torch.full((n,), 3.0, device=DEV, dtype=torch.bfloat16)
    keep = [t.clone() for t in ts + sc + [w]]
    zpp.adamw_step(*ts, step=5, scales=None if bits == 32 else ([sc[0]], [sc[1]]), weights=[w],
                   grad_scale=torch.tensor([c], device=DEV), **HP)
    for a, b in zip(ts + sc + [w], keep):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors_equal_single_calls(bits):
    """More tensors than one launch takes, empty ones among them."""
    T, g_ = 1000, gen(7)
    sizes = [(i * 37) % 700 if i % 9 else 0 for i in range(T)]
    code = torch.float32 if bits == 32 else torch.float8_e4m3fn
    P = [normal(n, 0.02, g_) for n in sizes]
    G = [normal(n, 1e-3, g_) for n in sizes]
    M, V = ([torch.zeros(n, device=DEV).to(code) for n in sizes] for _ in range(2))
    a, b = ([torch.zeros(-(-n // BLOCK), device=DEV) for n in sizes] for _ in range(2))
    if bits == 8:
        check_fp8(P, G, M, V, a, b, 1, seed=9)
        return
    one = [[t.clone() for t in ts] for ts in (P, G, M, V)]
    zpp.adamw_step(P, G, M, V, step=1, **HP)
    for p, g, m, v in zip(*one):
        zpp.adamw_step(p, g, m, v, step=1, **HP)
    for ts, us in zip((P, M, V), (one[0], one[2], one[3])):
        assert all(torch.equal(x, y) for x, y in zip(ts, us))


def test_optimiser_follows_the_definition():
    """Ten clipped steps of the class against fp64, then a resumed copy takes the same
    eleventh step bit for bit. Errors add up over the steps: ten times one step's bound on p
    (and the drift of the states inside it) stays below 1e-6 of the step sizes here."""
    g_ = gen(8)
    sizes = (1000, 33, 4097)
    P = [normal(n, 0.02, g_) for n in sizes]
    W = [torch.empty(n, device=DEV, dtype=torch.bfloat16) for n in sizes]
    opt = zpp.AdamW(P, weights=W, **HP)
    p = [x.double() for x in P]
    m = [torch.zeros_like(x) for x in p]
    v = [torch.zeros_like(x) for x in p]
    for t in range(1, 11):
        G = [normal(n, 1.0, g_).bfloat16() for n in sizes]
        norm = opt.step(G, max_norm=0.5, pre_scale=0.25)
        total = 0.25 * math.sqrt(sum(float(g.double().square().sum()) for g in G))
        c = 0.25 * min(1.0, 0.5 / total)
        assert abs(float(norm[0]) - total) < 1e-5 * total and abs(float(norm[1]) - c) < 1e-5 * c
        for i in range(3):
            p[i], m[i], v[i] = reference(p[i], G[i], m[i], v[i], t, c)[:3]
    for i in range(3):
        assert float((P[i].double() - p[i]).abs().max()) < 1e-6
        assert torch.equal(W[i], P[i].bfloat16())
    saved = opt.state()
    again = zpp.AdamW([x.clone() for x in P], exp_avg=[x.clone() for x in saved["exp_avg"]],
                      exp_avg_sq=[x.clone() for x in saved["exp_avg_sq"]], step=saved["step"], **HP)
    opt.step(G)
    again.step(G)
    assert all(torch.equal(x, y) for x, y in zip(P, again.params))


def test_another_stream():
    n, g_ = 100_003, gen(9)
    p, g = normal(n, 0.02, g_), normal(n, 1e-3, g_)
    m, v = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    want = reference(p, g, m, v, 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        zpp.adamw_step(p, g, m, v, step=1, **HP)
        norm = zpp.grad_norm(g)
    s.synchronize()
    within(p, want[0], want[3], "p")
    assert abs(float(norm[0]) - float(g.double().norm())) < 1e-5 * float(norm[0])


# ------------------------------------------------------------------------ gradient norm
# The sum of n squares in fp32: at most 16384 elements enter a partial, each thread adds a
# 256th of them in turn and the rest is a tree, so the relative error of the sum is below
# (64 + 10 + 2) u, half of that for its root; 1e-5 is more than twice that.
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("sizes", [(1,), (0, 5), (16384,), (16385, 3, 0, 40_000), (5_000_011,)])
def test_grad_norm(dtype, sizes):
    g_ = gen(10)
    G = [normal(n, 0.1, g_).to(dtype) for n in sizes]
    want = math.sqrt(sum(float(g.double().square().sum()) for g in G))
    for max_norm in (None, 0.5 * want, 2 * want):
        norm, coef = zpp.grad_norm(G, max_norm=max_norm, pre_scale=-0.5).tolist()
        assert abs(norm - 0.5 * want) <= 1e-5 * want
        clip = 1.0 if max_norm is None else min(1.0, max_norm / (0.5 * want))
        assert abs(coef + 0.5 * clip) <= 1e-5


def test_grad_norm_is_deterministic_and_reads_unaligned_ends():
    base = normal(1_000_003, 1.0, gen(11)).bfloat16()
    for lo, hi in ((0, 1_000_003), (8, 1_000_001), (16, 17), (24, 24 + 16384)):
        g = base[lo:hi]
        a, b = zpp.grad_norm(g), zpp.grad_norm(g)
        assert torch.equal(a, b)
        assert abs(float(a[0]) / float(g.double().norm()) - 1) < 1e-5


def test_grad_norm_of_zeros_and_of_non_finite_gradients():
    assert zpp.grad_norm(torch.zeros(1000, device=DEV), max_norm=1.0).tolist() == [0.0, 1.0]
    for bad in (math.inf, -math.inf, math.nan):
        g = torch.ones(40_000, device=DEV)
        g[33_333] = bad
        norm, coef = zpp.grad_norm(g, max_norm=1.0).tolist()
        assert not math.isfinite(norm) and math.isnan(coef)
    # squares beyond fp32's range count as overflow
    assert math.isnan(float(zpp.grad_norm(torch.full((10,), 1e30, device=DEV))[1]))


def test_overflowed_step_is_skipped_end_to_end():
    p = torch.ones(1000, device=DEV)
    opt = zpp.AdamW([p], **HP)
    g = torch.ones(1000, device=DEV, dtype=torch.float16)
    g[7] = math.inf
    opt.step(g, max_norm=1.0)
    assert bool((p == 1).all()) and bool((opt.exp_avg[0] == 0).all())


def test_offsets_beyond_32_bits():
    """A shard of more than 2^32 elements: the first and the last of them."""
    n, g_ = (1 << 32) + 1003, gen(12)
    p = torch.ones(n, device=DEV)
    g = torch.zeros(n, device=DEV, dtype=torch.bfloat16)
    m, v = (torch.zeros(n, device=DEV, dtype=torch.uint8).view(torch.float8_e4m3fn) for _ in range(2))
    a, b = (torch.zeros(-(-n // BLOCK), device=DEV) for _ in range(2))
    ends = (slice(0, 1024), slice(n - 1003 - 768, n))  # whole blocks, from multiples of 256 on
    for e in ends:
        g[e] = normal(e.stop - e.start, 1e-3, g_).bfloat16()
    zpp.adamw_step(p, g, m, v, step=1, scales=([a], [b]), seed=3, **HP)
    for e in ends:
        k = e.stop - e.start
        zero = torch.zeros(k, device=DEV)
        want = reference(torch.ones(k, device=DEV), g[e], zero, zero, 1)
        within(p[e], want[0], want[3], "p")
        for codes, scale, x, draw in ((m, a, want[1], 0), (v, b, want[2].sqrt(), 16)):
            s = scale[e.start // BLOCK:].double().repeat_interleave(BLOCK)[:k]
            bits = bits_of(torch.arange(e.start, e.stop, device=DEV), 3, 1) >> draw & 65535
            y = x.abs() / s
            h = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -6))) - 3)
            q = (torch.floor(y / h + (bits.double() + 0.5) / 65536) * h).clamp(max=448.0)
            q = torch.where(y > 0, q, q) if draw == 0 else torch.where(y > 0, q.clamp(min=2.0 ** -9), q)
            off = codes[e].double().abs() != q
            assert int(off.sum()) <= 2  # (a value within fp32's error of the next grid point)
    middle = slice(n // 2, n // 2 + 1000)
    assert bool((v[middle].float() == 0).all()) and float(p[middle].max()) < 1.0
    del p, g, m, v
    total = torch.full(((1 << 32) + 77,), 0.5, device=DEV, dtype=torch.float16)
    norm = zpp.grad_norm(total)
    assert abs(float(norm[0]) / (0.5 * math.sqrt(total.numel())) - 1) < 1e-5


def test_in_a_cuda_graph():
    """Norm, clip factor and step captured once (the step's number is captured with it)."""
    n, g_ = 10_007, gen(13)
    p, m, v = torch.ones(n, device=DEV), torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    g = normal(n, 1.0, g_).bfloat16()
    out = torch.empty(2, device=DEV)

    def work():
        zpp.grad_norm(g, max_norm=1.0, out=out)
        zpp.adamw_step(p, g, m, v, step=1, grad_scale=out[1:], **HP)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for seed in (1, 2):
        for t, value in ((p, 1.0), (m, 0.0), (v, 0.0)):
            t.fill_(value)
        g.copy_(normal(n, 1.0, gen(seed)))
        graph.replay()
        got = [t.clone() for t in (out, p, m, v)]
        for t, value in ((p, 1.0), (m, 0.0), (v, 0.0)):
            t.fill_(value)
        work()
        assert all(torch.equal(x, y) for x, y in zip(got, (out, p, m, v)))


def test_steps_back_to_back_wait_for_each_other():
    """Fifty clipped steps without a synchronisation equal fifty with one after each."""
    n, g_ = 3_000_001, gen(14)
    G = [normal(n, 1.0, g_).half() for _ in range(3)]
    out = []
    for sync in (False, True):
        p = torch.ones(n, device=DEV)
        opt = zpp.AdamW([p], state_bits=8, seed=2, **HP)
        for t in range(50):
            norm = opt.step([G[t % 3]], max_norm=1.0)
            if sync:
                torch.cuda.synchronize()
        out.append((p, norm, opt.exp_avg[0].float(), opt.exp_avg_sq[0].float(), *opt.scales[0]))
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_empty_list_through_the_c_interface():
    out, work = torch.full((2,), 7.0, device=DEV), torch.empty(1, device=DEV)
    assert zb.zpp_grad_norm([], [], zb.ZPP_F32, 0.25, 1.0, work.data_ptr(), out.data_ptr()) == zb.ZPP_OK
    assert out.tolist() == [0.0, 0.25]


def test_moved_storage_is_seen_by_the_next_step():
    """A parameter given new storage between two steps."""
    p = torch.ones(1000, device=DEV)
    opt = zpp.AdamW([p], **HP)
    g = torch.ones(1000, device=DEV)
    opt.step(g)
    old = p.data
    p.data = torch.full((1000,), 5.0, device=DEV)
    keep = old.clone()
    opt.step(g)
    assert torch.equal(old, keep) and float((p - 5.0).abs().max()) > 1e-3
    p.data = torch.ones(999, device=DEV)
    with pytest.raises(ValueError, match="999 elements, expected 1000"):
        opt.step(g)
