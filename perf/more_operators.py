"""Cases of the fp8 products with a scale per block of 128, and of the Muon step.

Each case is one call as a training or serving program makes it, with its plain form in
elementary torch operations (fp32) beside it and its definition in 64 bits (``exact``).

quant   a matrix to e4m3 codes with a power-of-two scale for each row and 128 columns (tile 1,
        activations and gradients) or for each tile of 128 x 128 (weights); with ``both`` also
        its transpose, as a backward pass needs it.
matmul  y = a b^T (+ bias) from e4m3 codes with a scale per block of 128 along the sum; b has a
        scale per tile of 128 x 128 (a weight) or per row (a gradient's other factor).
linear  one training pass of a linear layer in fp8: y, the gradients of x and of the weight.
orth    Newton-Schulz products that make a matrix (or a list) nearly orthogonal.
muon    one Muon step over a list of matrices: momentum, orthogonalised update, fp32 masters.
"""
import math
import random

import torch

own = False

BLOCK = 128
TOP = 448.0  # the largest e4m3 value
NS_STEPS, NS_EPS = 5, 1e-7
NS_A, NS_B, NS_C = 3.4445, -4.7750, 2.0315
MOMENTUM, DECAY = 0.95, 0.1
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # One token's activations before a projection: launch and call latency.
        dict(name="quant token", op="quant", rows=1, cols=8192, tile=1, both=False, dtype="bf16"),
        # A micro-batch's activations, kept in both orientations for the backward pass.
        dict(name="quant batch", op="quant", rows=16384, cols=8192, tile=1, both=True,
             dtype="bf16"),
        # The fp32 master of a hidden-8192 layer's 24576 x 8192 matrix after an optimiser step.
        dict(name="quant weight", op="quant", rows=24576, cols=8192, tile=128, both=True,
             dtype="f32"),
        # One token through that matrix: bound by reading the codes.
        dict(name="matmul token", op="matmul", m=1, n=24576, k=8192, btile=128, out="bf16",
             bias=False, order="blocks"),
        # 77 sequences decoded together: odd vocabulary, odd width, fp32 logits.
        dict(name="matmul odd", op="matmul", m=77, n=50001, k=1003, btile=128, out="f32",
             bias=True, order="rows"),
        # A prompt of 8192 tokens through the QKV projection.
        dict(name="matmul prompt", op="matmul", m=8192, n=24576, k=8192, btile=128, out="bf16",
             bias=False, order="blocks"),
        # A small model's layer and micro-batch: seven short kernels.
        dict(name="linear small", op="linear", tokens=1024, n=1024, k=1024, dtype="bf16",
             weight="bf16"),
        # A square projection of a hidden-8192 layer.
        dict(name="linear layer", op="linear", tokens=8192, n=8192, k=8192, dtype="bf16",
             weight="f32"),
        # One small matrix: fifteen dependent products, latency.
        dict(name="orth small", op="orth", count=1, rows=256, cols=1024, dtype="bf16"),
        # The MLP matrix of a hidden-4096 layer.
        dict(name="orth large", op="orth", count=1, rows=4096, cols=16384, dtype="bf16"),
        # Four layers of a hidden-1024 model: 24 matrices of three shapes, clipped.
        dict(name="muon layers", op="muon", shapes="16x1024x1024 4x4096x1024 4x1024x4096",
             grad="bf16", weight="bf16", adjust="match_rms_adamw", lr=2e-4, nesterov=True,
             clip=True),
        # A hidden-4096 layer's share of one rank.
        dict(name="muon large", op="muon", shapes="2x4096x4096 1x16384x4096", grad="f32",
             weight="none", adjust="original", lr=2e-3, nesterov=True, clip=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A size of the range: any number, or a multiple of 64."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.4 else max(64, n // 64 * 64)


def draw(rng):
    op = rng.choice(("quant", "matmul", "matmul", "linear", "orth", "muon"))
    if op == "quant":
        cols = _size(rng, 64, 32768)
        rows = min(_log(rng, 1, 32768), 134_000_000 // cols)
        return dict(op=op, rows=rows, cols=cols, tile=rng.choice((1, 1, 128)),
                    both=rng.random() < 0.5, dtype=rng.choice(("bf16", "f16", "f32")))
    if op == "matmul":
        n, k = _size(rng, 64, 50_000), _size(rng, 64, 20_000)
        m = min(_log(rng, 1, 16384), max(1, 1_600_000_000_000 // (n * k)))
        return dict(op=op, m=m, n=n, k=k, btile=rng.choice((128, 128, 1)),
                    out=rng.choice(("bf16", "f16", "f32")), bias=rng.random() < 0.3,
                    order=rng.choice(("blocks", "rows")))
    if op == "linear":
        n, k = _size(rng, 64, 10_000), _size(rng, 64, 10_000)
        tokens = min(_log(rng, 8, 16384), max(8, 400_000_000_000 // (n * k)))
        return dict(op=op, tokens=tokens, n=n, k=k, dtype=rng.choice(("bf16", "f16")),
                    weight=rng.choice(("bf16", "f16", "f32")))
    if op == "orth":
        rows, cols = _size(rng, 32, 6000), _size(rng, 32, 6000)
        count = min(rng.choice((1, 1, 2, 5, 12)), max(1, 40_000_000 // (rows * cols)))
        return dict(op=op, count=count, rows=rows, cols=cols, dtype=rng.choice(("bf16", "f16")))
    shapes, left = [], 40_000_000
    for _ in range(rng.choice((1, 2, 3, 4))):
        rows, cols = _size(rng, 32, 4096), _size(rng, 32, 4096)
        count = min(rng.choice((1, 1, 2, 6)), left // (rows * cols))
        if count:
            shapes.append(f"{count}x{rows}x{cols}")
            left -= count * rows * cols
    adjust, lr = rng.choice((("match_rms_adamw", 2e-4), ("original", 2e-3)))
    return dict(op=op, shapes=" ".join(shapes), grad=rng.choice(("f32", "bf16", "f16")),
                weight=rng.choice(("none", "bf16", "f16")), adjust=adjust, lr=lr,
                nesterov=rng.random() < 0.7, clip=rng.random() < 0.5)


def _shapes(case):
    """[(count, rows, cols)] of a list of matrices."""
    return [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split()]


# ------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _activations(gen, rows, cols, dtype):
    """Normal values; channels of unequal size, a few of them far larger."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    size = torch.exp(0.5 * torch.randn(cols, generator=gen, device="cuda"))
    size[::97] *= 20.0
    return (x * size).to(dtype)


def _gradient(gen, rows, cols, dtype):
    """Heavy-tailed, as gradients are."""
    u = torch.rand(rows, cols, generator=gen, device="cuda") - 0.5
    return (-1e-4 * u.sign() * torch.log1p(-2.0 * u.abs().clamp(max=0.4999999))).to(dtype)


def _update(gen, count, rows, cols):
    """A stack of averaged gradients: a few strong directions over noise."""
    r = max(1, min(rows, cols) // 64)
    left = torch.randn(count, rows, r, generator=gen, device="cuda")
    right = torch.randn(count, r, cols, generator=gen, device="cuda")
    noise = torch.randn(count, rows, cols, generator=gen, device="cuda")
    return 1e-4 * (noise + (2.0 / math.sqrt(r)) * torch.matmul(left, right))


def _coded(x, tile):
    """x as another program's e4m3 codes, rows at multiples of 16 bytes, and scales amax / 448."""
    rows, cols = x.shape
    down, across = -(-rows // tile), -(-cols // BLOCK)
    wide = torch.zeros(down * tile, across * BLOCK, device="cuda")
    wide[:rows, :cols] = x
    blocks = wide.view(down, tile, across, BLOCK)
    scales = (blocks.abs().amax((1, 3)) / TOP).clamp(min=1e-30)
    codes = (blocks / scales[:, None, :, None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn)
    apart = -(-cols // 16) * 16
    held = codes.view(torch.uint8).view(down * tile, across * BLOCK)[:rows, :apart].contiguous()
    return held.view(torch.float8_e4m3fn)[:, :cols], scales


def prepare(case, seed):
    gen, op = _gen(seed), case["op"]
    s = dict(case=case)
    if op == "quant":
        dt = DTYPES[case["dtype"]]
        if case["tile"] == 1:
            s["x"] = _activations(gen, case["rows"], case["cols"], dt)
        else:
            s["x"] = (0.02 * torch.randn(case["rows"], case["cols"], generator=gen,
                                         device="cuda")).to(dt)
        return s
    if op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"], a_scales = _coded(_activations(gen, m, k, torch.float32), 1)
        s["a_scales"] = a_scales.t().contiguous().t() if case["order"] == "blocks" else a_scales
        w = 0.02 * torch.randn(n, k, generator=gen, device="cuda")
        s["b"], b_scales = _coded(w, case["btile"])
        if case["btile"] == 1 and case["order"] == "blocks":
            b_scales = b_scales.t().contiguous().t()
        s["b_scales"] = b_scales
        s["out"] = DTYPES[case["out"]]
        s["bias"] = None
        if case["bias"]:
            s["bias"] = torch.randn(n, generator=gen, device="cuda").to(s["out"])
        return s
    if op == "linear":
        dt = DTYPES[case["dtype"]]
        s["x"] = _activations(gen, case["tokens"], case["k"], dt).requires_grad_()
        s["w"] = (0.02 * torch.randn(case["n"], case["k"], generator=gen, device="cuda")).to(
            DTYPES[case["weight"]]).requires_grad_()
        s["dy"] = _gradient(gen, case["tokens"], case["n"], dt)
        return s
    if op == "orth":
        s["stack"] = _update(gen, case["count"], case["rows"], case["cols"]).to(
            DTYPES[case["dtype"]])
        s["list"] = list(s["stack"])
        return s
    shapes = _shapes(case)
    randn = lambda *v: torch.randn(*v, generator=gen, device="cuda")  # noqa: E731
    s["p"] = [0.02 * randn(*v) for v in shapes]
    s["g"] = [(0.2 * _update(gen, *v) + 1e-4 * randn(*v)).to(DTYPES[case["grad"]])
              for v in shapes]
    s["m"] = [_update(gen, *v) for v in shapes]
    weight = case["weight"]
    s["w"] = None if weight == "none" else [torch.zeros(v, dtype=DTYPES[weight], device="cuda")
                                            for v in shapes]
    total = sum(c * rows * cols for c, rows, cols in shapes)
    # about half the norm that these gradients have, so that the clip acts
    s["max_norm"] = 0.5 * 1.1e-4 * math.sqrt(total) if case["clip"] else None
    s["grads"] = [g for stack in s["g"] for g in stack]
    if own:
        import quantized_zero_communication_gb300 as zpp
        each = lambda stacks: [t for stack in stacks for t in stack]  # noqa: E731
        s["opt"] = zpp.Muon(each(s["p"]), lr=case["lr"], momentum=MOMENTUM,
                            weight_decay=DECAY, nesterov=case["nesterov"],
                            coefficients=(NS_A, NS_B, NS_C), steps=NS_STEPS, eps=NS_EPS,
                            adjust=case["adjust"], buffers=each(s["m"]),
                            weights=None if s["w"] is None else each(s["w"]))
    return s


# --------------------------------------------------------------------------- the passes
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    return {"quant": _quant_plain, "matmul": _matmul_plain, "linear": _linear_plain,
            "orth": _orth_plain, "muon": _muon_plain}[op](s)


def _own(s, op):
    import quantized_zero_communication_gb300 as zpp
    c = s["case"]
    if op == "quant":
        return list(zpp.quant_fp8(s["x"], c["tile"], transposed=c["both"]))
    if op == "matmul":
        return zpp.matmul_fp8(s["a"], s["a_scales"], s["b"], s["b_scales"], bias=s["bias"],
                              dtype=s["out"])
    if op == "linear":
        y = zpp.linear_fp8(s["x"], s["w"])
        dx, dw = torch.autograd.grad(y, (s["x"], s["w"]), s["dy"])
        return [y.detach(), dx, dw]
    if op == "orth":
        return zpp.orthogonalize(s["list"], steps=NS_STEPS, coefficients=(NS_A, NS_B, NS_C),
                                 eps=NS_EPS)
    norm = s["opt"].step(s["grads"], max_norm=s["max_norm"])
    return _stepped(s, norm)


def _scale_of(amax):
    """The smallest power of two that amax / scale <= 448 holds for, at least 2^-126; 0 for 0."""
    part, power = torch.frexp(amax)  # amax = part 2^power, 1/2 <= part < 1; 448 = 7/8 2^9
    power = power - torch.where(part <= 0.875, 9, 8)
    scale = torch.ldexp(torch.ones_like(amax), power.clamp(min=-126))
    return torch.where(amax > 0, scale, torch.zeros_like(amax))


def _quantised(x, down):
    """x in fp32 -> (values as e4m3 codes, scales) with a scale for each `down` rows and 128
    columns; what is beyond the edge counts as 0."""
    rows, cols = x.shape
    d, a = -(-rows // down), -(-cols // BLOCK)
    wide = x
    if d * down != rows or a * BLOCK != cols:
        wide = torch.zeros(d * down, a * BLOCK, device="cuda")
        wide[:rows, :cols] = x
    blocks = wide.view(d, down, a, BLOCK)
    scales = _scale_of(blocks.abs().amax((1, 3)))
    inv = torch.where(scales > 0, 1.0 / scales, torch.zeros_like(scales))
    codes = (blocks * inv[:, None, :, None]).to(torch.float8_e4m3fn)
    return codes.view(d * down, a * BLOCK)[:rows, :cols], scales


def _quant_plain(s):
    tile = s["case"]["tile"]
    x = s["x"].float()
    out = list(_quantised(x, tile))
    if s["case"]["both"] and tile == 1:
        out += _quantised(x.t(), 1)
    elif s["case"]["both"]:
        out += [out[0].view(torch.uint8).t().contiguous().view(torch.float8_e4m3fn), out[1].t()]
    return out


def _value(codes, scales, down):
    """The values that codes stand for, fp32."""
    rows, cols = codes.shape
    each = scales.repeat_interleave(BLOCK, 1)[:, :cols]
    return codes.float() * (each if down == 1 else each.repeat_interleave(down, 0)[:rows])


def _matmul_plain(s):
    a = _value(s["a"], s["a_scales"], 1)
    b = _value(s["b"], s["b_scales"], s["case"]["btile"])
    y = torch.matmul(a, b.t())
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["out"])


def _linear_plain(s):
    x, w, dy = s["x"].detach().float(), s["w"].detach().float(), s["dy"].float()
    wq = _value(*_quantised(w, BLOCK), BLOCK)
    y = torch.matmul(_value(*_quantised(x, 1), 1), wq.t())
    dx = torch.matmul(_value(*_quantised(dy, 1), 1), wq)
    dw = torch.matmul(_value(*_quantised(dy.t(), 1), 1), _value(*_quantised(x.t(), 1), 1).t())
    return [y.to(s["x"].dtype), dx.to(s["x"].dtype), dw.to(s["w"].dtype)]


def _newton_schulz(x):
    """A stack of matrices, fp32 -> the same, nearly orthogonal."""
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2)
    x = x / (x * x).sum((1, 2), keepdim=True).sqrt().clamp(min=NS_EPS)
    for _ in range(NS_STEPS):
        a = torch.matmul(x, x.transpose(1, 2))
        b = NS_B * a + NS_C * torch.matmul(a, a)
        x = NS_A * x + torch.matmul(b, x)
    return x.transpose(1, 2) if tall else x


def _orth_plain(s):
    return list(_newton_schulz(s["stack"].float()).to(s["stack"].dtype))


def _adjusted(case, rows, cols):
    """The learning rate of a matrix."""
    if case["adjust"] == "original":
        return case["lr"] * math.sqrt(max(1.0, rows / cols))
    return case["lr"] * 0.2 * math.sqrt(max(rows, cols))


def _stepped(s, norm):
    out = dict(p=s["p"], m=s["m"])
    if s["w"] is not None:
        out["w"] = s["w"]
    if norm is not None:
        out["norm"] = norm
    return out


def _muon_plain(s):
    c = s["case"]
    norm = None
    if c["clip"]:
        total = sum((g.float() * g.float()).sum() for g in s["g"]).sqrt()
        norm = torch.stack([total, (s["max_norm"] / total).clamp(max=1.0)])
    for i, (p, g, m) in enumerate(zip(s["p"], s["g"], s["m"])):
        g = g.float()
        if norm is not None:
            g = g * norm[1]
        m.copy_(MOMENTUM * m + (1.0 - MOMENTUM) * g)
        u = (1.0 - MOMENTUM) * g + MOMENTUM * m if c["nesterov"] else m
        lr = _adjusted(c, p.shape[1], p.shape[2])
        p.copy_(p * (1.0 - c["lr"] * DECAY) - lr * _newton_schulz(u))
        if s["w"] is not None:
            s["w"][i].copy_(p)
    return _stepped(s, norm)


# ---------------------------------------------------------------------------- the work
def _quant_bytes(rows, cols, tile, both, size):
    scales = 4.0 * -(-rows // tile) * -(-cols // BLOCK)
    if both and tile == 1:  # (a tile's scale is that of the transpose too)
        scales += 4.0 * cols * -(-rows // BLOCK)
    return rows * cols * (size + (2.0 if both else 1.0)) + scales


def _ns_flops(rows, cols):
    """Two of a step's three products are symmetric: half of them is enough."""
    m, n = min(rows, cols), max(rows, cols)
    return NS_STEPS * (3.0 * m * m * n + 1.0 * m * m * m)


def work(case):
    op = case["op"]
    size = lambda kind: 4 if kind == "f32" else 2  # noqa: E731
    if op == "quant":
        n = case["rows"] * case["cols"]
        return dict(bytes=_quant_bytes(case["rows"], case["cols"], case["tile"], case["both"],
                                       size(case["dtype"])), flops=4.0 * n)
    if op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        across, y = -(-k // BLOCK), size(case["out"])
        return dict(bytes=(m + n) * k + 4.0 * across * (m + -(-n // case["btile"])) + m * n * y
                    + (n * y if case["bias"] else 0), flops=2.0 * m * n * k)
    if op == "linear":
        t, n, k = case["tokens"], case["n"], case["k"]
        return dict(bytes=t * (4.0 * k + 4.0 * n) + 2.0 * n * k * size(case["weight"]),
                    flops=6.0 * t * n * k)
    if op == "orth":
        rows, cols, count = case["rows"], case["cols"], case["count"]
        return dict(bytes=4.0 * count * rows * cols, flops=count * _ns_flops(rows, cols))
    total = sum(c * rows * cols for c, rows, cols in _shapes(case))
    w = 0 if case["weight"] == "none" else 2
    return dict(bytes=total * (16.0 + size(case["grad"]) + w),
                flops=sum(c * _ns_flops(rows, cols) for c, rows, cols in _shapes(case)))


# ------------------------------------------------------------------------- in 64 bits
def _grid(x, down):
    """(e4m3 values of x / scale, scales, values that they stand for), all in 64 bits: round to
    nearest, ties to even, on the spacing 2^(floor(log2 |v|) - 3), 2^-9 below 2^-6."""
    rows, cols = x.shape
    top = torch.zeros(-(-rows // down) * down, -(-cols // BLOCK) * BLOCK, dtype=torch.float64,
                      device="cuda")
    top[:rows, :cols] = x.abs()
    top = top.unfold(0, down, down).unfold(1, BLOCK, BLOCK).amax((2, 3))
    power = torch.ceil(torch.log2(top / TOP))
    # (a logarithm may be off by its last bit: the power is checked on both sides)
    power = torch.where(top > TOP * torch.exp2(power), power + 1, power)
    power = torch.where(top <= TOP * torch.exp2(power - 1), power - 1, power).clamp(min=-126)
    scales = torch.where(top > 0, torch.exp2(power), torch.zeros_like(top))
    full = torch.kron(scales, torch.ones(down, BLOCK, dtype=torch.float64, device="cuda"))
    full = full[:rows, :cols]
    v = torch.where(full > 0, x / full, torch.zeros_like(x))
    h = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    v = torch.round(v / h) * h
    return v, scales, v * full


def _ns_exact(x):
    x = x.double()
    wide = x if x.shape[0] <= x.shape[1] else x.T
    y = wide / max(float(torch.linalg.vector_norm(wide)), NS_EPS)
    eye = torch.eye(y.shape[0], dtype=torch.float64, device="cuda")
    for _ in range(NS_STEPS):
        gram = y @ y.T
        y = torch.addmm(NS_B * gram, gram, gram, alpha=NS_C).add_(eye, alpha=NS_A) @ y
    return y if x.shape[0] <= x.shape[1] else y.T


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        x = s["x"].double()
        v, scales, _ = _grid(x, case["tile"])
        out = [v, scales]
        if case["both"]:
            out += list(_grid(x.T, 1)[:2]) if case["tile"] == 1 else [v.T, scales.T]
        return out
    if op == "matmul":
        def held(codes, scales, down):
            ones = torch.ones(down, BLOCK, dtype=torch.float64, device="cuda")
            each = torch.kron(scales.double().contiguous(), ones)
            return codes.to(torch.float64) * each[:codes.shape[0], :codes.shape[1]]
        y = held(s["a"], s["a_scales"], 1) @ held(s["b"], s["b_scales"], case["btile"]).T
        return y if s["bias"] is None else y + s["bias"].double()
    if op == "linear":
        x, w, dy = (s[v].detach().double() for v in ("x", "w", "dy"))
        wq = _grid(w, BLOCK)[2]
        y = _grid(x, 1)[2] @ wq.T
        dx = _grid(dy, 1)[2] @ wq
        del wq
        return [y, dx, _grid(dy.T, 1)[2] @ _grid(x.T, 1)[2].T]
    if op == "orth":
        return [_ns_exact(x) for x in s["list"]]
    clip, norm = 1.0, None
    if case["clip"]:
        total = math.sqrt(sum(float(g.double().pow(2).sum()) for g in s["g"]))
        clip = min(1.0, s["max_norm"] / total)
        norm = torch.tensor([total, clip], dtype=torch.float64, device="cuda")
    out = dict(p=[], m=[])
    for p, g, m in zip(s["p"], s["g"], s["m"]):
        g = g.double() * clip
        m = torch.lerp(g, m.double(), MOMENTUM)
        u = torch.lerp(g, m, MOMENTUM) if case["nesterov"] else m
        lr = _adjusted(case, p.shape[1], p.shape[2])
        o = torch.stack([_ns_exact(v) for v in u])
        out["p"].append(p.double() * (1 - case["lr"] * DECAY) - lr * o)
        out["m"].append(m)
    if s["w"] is not None:
        out["w"] = out["p"]
    if norm is not None:
        out["norm"] = norm
    return out
