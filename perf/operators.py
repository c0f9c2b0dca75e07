"""Cases of the optimiser step, the gradient norm and the product with block-quantised weights.

Each case is one call as a training or serving program makes it, with its plain form in
elementary torch operations (fp32) beside it and its definition in 64 bits (``exact``).

adamw   one step over a list of tensors, fp32 master weights, states in fp32 or in fp8
        (e4m3 with one fp32 scale per 256 elements, rounded stochastically from a seed).
        The shards lie in flat buffers, as a data-parallel partition holds them, each tensor
        starting at a multiple of ``align`` elements; with ``clip`` the step first takes
        the global gradient norm.
norm    the global gradient norm and the factor that clips it.
matvec  y = x W^T (+ bias) with W held as INT4 / INT8 codes and a scale per `block` elements.
"""
import math
import random

import torch

own = False

STATE_BLOCK = 256  # elements per fp8 state scale
BETA1, BETA2, EPS, LR, DECAY = 0.9, 0.999, 1e-8, 1e-4, 0.1
STEP0 = 1000  # steps taken before the measured one
SEED0 = 77    # of the stochastic rounding
MASK32 = 0xFFFFFFFF
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # One layer-norm weight of a small model: launch and call latency.
        dict(name="adamw32 one vector", op="adamw", state=32, total=1024, tensors=1, align=8,
             grad="bf16", weight="bf16", clip=False),
        # An unflattened small model: many tensors of unequal, odd sizes, clipped.
        dict(name="adamw32 list", op="adamw", state=32, total=12_000_000, tensors=150, align=8,
             grad="f32", weight="bf16", clip=True),
        # A flat shard: the 8192 x 24576 matrix of a hidden-8192 layer.
        dict(name="adamw32 shard", op="adamw", state=32, total=201_326_592, tensors=1, align=8,
             grad="bf16", weight="bf16", clip=False),
        # One rank's bucket of a hidden-1024 model as 13 tensors, fp8 states, clipped.
        dict(name="adamw8 bucket", op="adamw", state=8, total=16_777_216, tensors=13, align=256,
             grad="f16", weight="f16", clip=True),
        # The largest flat shard (a 32768 x 8192 matrix), fp8 states.
        dict(name="adamw8 shard", op="adamw", state=8, total=268_435_456, tensors=1, align=256,
             grad="bf16", weight="bf16", clip=False),
        # The norm of a small fp32 list, and of a large bf16 gradient bucket.
        dict(name="norm list", op="norm", total=1_000_003, tensors=40, align=8, grad="f32"),
        dict(name="norm bucket", op="norm", total=536_870_912, tensors=13, align=8, grad="bf16"),
        # One token through a small square projection: latency.
        dict(name="matvec4 small", op="matvec", rows=1024, cols=1024, block=64, bits=4, vecs=1,
             dtype="f16", out="f16", bias=True),
        # One token through the QKV projection of a hidden-8192 layer.
        dict(name="matvec4 qkv", op="matvec", rows=24576, cols=8192, block=128, bits=4, vecs=1,
             dtype="bf16", out="bf16", bias=False),
        # Eight sequences decoded together through an MLP matrix, fp32 out.
        dict(name="matvec4 batch", op="matvec", rows=8192, cols=32768, block=256, bits=4, vecs=8,
             dtype="bf16", out="f32", bias=False),
        # One token, INT8 codes with the block of the weight all-gather.
        dict(name="matvec8 square", op="matvec", rows=8192, cols=8192, block=2048, bits=8, vecs=1,
             dtype="f16", out="f16", bias=False),
        # An odd vocabulary and an odd width: blocks run across the rows.
        dict(name="matvec4 odd", op="matvec", rows=50001, cols=1003, block=64, bits=4, vecs=3,
             dtype="f16", out="f32", bias=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("adamw", "adamw", "norm", "matvec", "matvec"))
    if op == "adamw":
        state, total = rng.choice((32, 8)), _log(rng, 1000, 200_000_000)
        return dict(op=op, state=state, total=total, tensors=min(_log(rng, 1, 300), max(1, total // 64)),
                    align=256 if state == 8 else rng.choice((8, 256)),
                    grad=rng.choice(("f32", "bf16", "f16")),
                    weight=rng.choice(("none", "bf16", "f16")), clip=rng.random() < 0.5)
    if op == "norm":
        total = _log(rng, 1000, 400_000_000)
        return dict(op=op, total=total, tensors=min(_log(rng, 1, 300), max(1, total // 64)),
                    align=rng.choice((8, 256)), grad=rng.choice(("f32", "bf16", "f16")))
    block = rng.choice((64, 128, 256, 512, 1024, 2048, 4096))
    rows, cols = _log(rng, 100, 40_000), _log(rng, 256, 30_000)
    kind = rng.choice(("whole", "whole", "whole", "even", "odd"))
    if kind == "whole":  # every block inside one row
        cols = max(block, cols // block * block)
    elif kind == "even":
        cols = max(16, cols // 16 * 16)
    rows = max(1, min(rows, 200_000_000 // cols))
    return dict(op=op, rows=rows, cols=cols, block=block, bits=rng.choice((4, 4, 8)),
                vecs=rng.choice((1, 1, 1, 2, 3, 4, 5, 8, 13, 16)), dtype=rng.choice(("bf16", "f16")),
                out=rng.choice(("same", "f32")), bias=rng.random() < 0.3)


def _sizes(case):
    """Element counts of the case's tensors: unequal, odd ones among them, each at least 1."""
    n, total = case["tensors"], case["total"]
    rng = random.Random(total * 31 + n)
    share = [math.exp(rng.gauss(0.0, 1.5)) for _ in range(n)]
    whole = sum(share)
    sizes = [max(1, int(total * s / whole)) for s in share]
    sizes[-1] = max(1, sizes[-1] + total - sum(sizes))
    return sizes


def _offsets(case):
    """(offset of every tensor in the flat buffer, the buffer's length)."""
    at, a = [], case["align"]
    end = 0
    for n in _sizes(case):
        at.append(end)
        end += -(-n // a) * a
    return at, end


# ------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _views(flat, at, sizes):
    return [flat[o:o + n] for o, n in zip(at, sizes)]


def _fill(n_flat, at, sizes, make, dtype):
    """A flat buffer whose tensors hold make(n) and whose gaps hold zeros."""
    flat = make(n_flat).to(dtype)
    for i, (o, n) in enumerate(zip(at, sizes)):
        flat[o + n:at[i + 1] if i + 1 < len(at) else n_flat] = 0
    return flat


def _grads(case, gen, at, sizes, n_flat):
    def make(n):  # heavy-tailed, as gradients are
        u = torch.rand(n, generator=gen, device="cuda") - 0.5
        return -1e-4 * u.sign() * torch.log1p(-2.0 * u.abs().clamp(max=0.4999999))
    return _fill(n_flat, at, sizes, make, DTYPES[case["grad"]])


def prepare(case, seed):
    gen = _gen(seed)
    s = dict(case=case)
    if case["op"] == "matvec":
        rows, cols, block, bits = case["rows"], case["cols"], case["block"], case["bits"]
        n, qmax = rows * cols, 2 ** (bits - 1) - 1
        blocks = -(-n // block)
        w = torch.zeros(blocks * block, device="cuda")
        w[:n].normal_(0.0, 0.02, generator=gen)
        w = w.view(blocks, block)
        amax = w.abs().amax(1)
        q = torch.round(w * (qmax / amax)[:, None]).to(torch.int8).view(-1)[:n]
        s["scales"] = amax / qmax
        if bits == 4:
            if n % 2:
                q = torch.cat([q, q.new_zeros(1)])
            q = (q[0::2] & 15) | (q[1::2] << 4)
        s["codes"] = q.view(torch.uint8)
        dt = DTYPES[case["dtype"]]
        s["x"] = torch.randn(case["vecs"], cols, generator=gen, device="cuda").to(dt)
        s["bias"] = torch.randn(rows, generator=gen, device="cuda").to(dt) if case["bias"] else None
        s["out"] = dt if case["out"] == "same" else DTYPES[case["out"]]
        return s
    sizes, (at, n_flat) = _sizes(case), _offsets(case)
    g = _grads(case, gen, at, sizes, n_flat)
    s.update(g=g, grads=_views(g, at, sizes))
    # about half the norm that these gradients have, so that the clip acts
    s["max_norm"] = 0.5 * 1.4e-4 * math.sqrt(case["total"])
    if case["op"] == "norm":
        return s
    randn = lambda n: torch.randn(n, generator=gen, device="cuda")  # noqa: E731
    p = _fill(n_flat, at, sizes, lambda n: 0.02 * randn(n), torch.float32)
    m = _fill(n_flat, at, sizes, lambda n: 3e-5 * randn(n), torch.float32)
    r = _fill(n_flat, at, sizes, lambda n: 1.4e-4 * (0.3 + randn(n).abs()), torch.float32)
    s.update(p=p, step=STEP0)
    if case["state"] == 8:
        def encode(x):
            x = x.view(-1, STATE_BLOCK)
            scale = x.abs().amax(1) / 448.0
            return (x / scale[:, None].clamp(min=1e-30)).to(torch.float8_e4m3fn).view(-1), scale
        s["m"], s["ms"] = encode(m)
        s["v"], s["vs"] = encode(r)  # the root of the second moment is what is held
    else:
        s["m"], s["v"] = m, r * r
    weight = case["weight"]
    s["w"] = None if weight == "none" else torch.zeros(n_flat, dtype=DTYPES[weight], device="cuda")
    if own:
        import quantized_zero_communication_gb300 as zpp
        scaled = case["state"] == 8
        cut = [-(-n // STATE_BLOCK) for n in sizes]
        of = [o // STATE_BLOCK for o in at]
        s["opt"] = zpp.AdamW(
            _views(p, at, sizes), lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY,
            state_bits=case["state"], exp_avg=_views(s["m"], at, sizes),
            exp_avg_sq=_views(s["v"], at, sizes),
            scales=(_views(s["ms"], of, cut), _views(s["vs"], of, cut)) if scaled else None,
            weights=None if s["w"] is None else _views(s["w"], at, sizes), step=STEP0, seed=SEED0)
    return s


# --------------------------------------------------------------------------- the passes
def run(s):
    op = s["case"]["op"]
    if op == "matvec":
        return _matvec_own(s) if own else _matvec_plain(s)
    if op == "norm":
        if own:
            import quantized_zero_communication_gb300 as zpp
            return zpp.grad_norm(s["grads"], max_norm=s["max_norm"])
        return _norm_plain(s["g"], s["max_norm"])
    return _adamw_own(s) if own else _adamw_plain(s)


def _matvec_own(s):
    import quantized_zero_communication_gb300 as zpp
    c = s["case"]
    return zpp.matvec_blockwise(s["codes"], s["scales"], s["x"], c["rows"], c["block"], c["bits"],
                                bias=s["bias"], dtype=s["out"])


def _codes(s):
    """The signed codes, one int8 per weight."""
    c = s["case"]
    if c["bits"] == 8:
        return s["codes"].view(torch.int8)
    b = s["codes"].view(torch.int8)
    return torch.stack([(b << 4) >> 4, b >> 4], 1).view(-1)[:c["rows"] * c["cols"]]


def _matvec_plain(s):
    c = s["case"]
    n, block = c["rows"] * c["cols"], c["block"]
    q = _codes(s).float()
    whole = n // block * block
    w = torch.empty(n, device="cuda")
    w[:whole] = (q[:whole].view(-1, block) * s["scales"][:n // block, None]).view(-1)
    if whole < n:
        w[whole:] = q[whole:] * s["scales"][-1]
    y = torch.matmul(s["x"].float(), w.view(c["rows"], c["cols"]).t())
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["out"])


def _norm_plain(g, max_norm):
    g = g.float()
    norm = (g * g).sum().sqrt()
    coef = torch.where(norm > max_norm, max_norm / norm, torch.ones_like(norm))
    return torch.stack([norm, coef])


def _adamw_own(s):
    norm = s["opt"].step(s["grads"], max_norm=s["max_norm"] if s["case"]["clip"] else None)
    return _updated(s, norm)


def _updated(s, norm):
    out = dict(p=s["p"], m=s["m"], v=s["v"])
    if s["case"]["state"] == 8:
        out.update(ms=s["ms"], vs=s["vs"])
    if s["w"] is not None:
        out["w"] = s["w"]
    if norm is not None:
        out["norm"] = norm
    return out


def _random_bits(n, step):
    """32 random bits for every element: a hash of its number in the list (blocks of 256
    counted through the tensors), the seed and the step."""
    key = ((SEED0 * 0x9E3779B9) ^ (step * 0x510E527F)) & MASK32
    x = torch.arange(n, device="cuda")
    x = ((x & MASK32) * 0x9E3779B9 + (x >> 32) * 0xA54FF53B + key) & MASK32
    x = ((x ^ (x >> 16)) * 0xBB67AE85 + key) & MASK32
    x = ((x ^ (x >> 15)) * 0x9B05688D) & MASK32
    return x ^ (x >> 16)


def _encode(x, bits16, keep):
    """x in blocks of 256 -> (e4m3 values of x / scale rounded stochastically, scales).
    `keep`: a value above zero stays above zero."""
    x = x.view(-1, STATE_BLOCK)
    a = x.abs()
    scale = a.amax(1) / 448.0
    inv = torch.where(scale > 0, 448.0 / a.amax(1), torch.zeros_like(scale))
    a = (a * inv[:, None]).view(-1)
    low = a < 2.0 ** -6  # there the grid is that of the range above, shifted
    b = torch.where(low, a + 2.0 ** -6, a).view(torch.int32)
    b = (b + (bits16 * 16 + 8).to(torch.int32)) & ~0xFFFFF
    b = b.view(torch.float32)
    b = torch.where(low, b - 2.0 ** -6, b).clamp(max=448.0)
    if keep:
        b = torch.where(a > 0, b.clamp(min=2.0 ** -9), b)
    return torch.where(x.view(-1) < 0, -b, b).to(torch.float8_e4m3fn), scale


def _adamw_plain(s):
    c = s["case"]
    s["step"] += 1
    t = s["step"]
    g = s["g"].float()
    norm = None
    if c["clip"]:
        norm = _norm_plain(s["g"], s["max_norm"])
        g = g * norm[1]
    if c["state"] == 8:
        n = g.numel()
        m = (s["m"].float().view(-1, STATE_BLOCK) * s["ms"][:, None]).view(n)
        r = (s["v"].float().view(-1, STATE_BLOCK) * s["vs"][:, None]).view(n)
        v = r * r
    else:
        m, v = s["m"], s["v"]
    m = BETA1 * m + (1.0 - BETA1) * g
    v = BETA2 * v + (1.0 - BETA2) * (g * g)
    root = v.sqrt()
    denom = root / math.sqrt(1.0 - BETA2 ** t) + EPS
    p = s["p"] * (1.0 - LR * DECAY) - (LR / (1.0 - BETA1 ** t)) * (m / denom)
    s["p"].copy_(p)
    if c["state"] == 8:
        bits = _random_bits(g.numel(), t)
        for name, x, b, keep in (("m", m, bits & 0xFFFF, False), ("v", root, bits >> 16, True)):
            q, scale = _encode(x, b, keep)
            s[name].copy_(q)
            s[name + "s"].copy_(scale)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    if s["w"] is not None:
        s["w"].copy_(p)
    return _updated(s, norm)


# ---------------------------------------------------------------------------- the work
def work(case):
    if case["op"] == "matvec":
        n = case["rows"] * case["cols"]
        x = 2
        y = 4 if case["out"] == "f32" else 2
        return dict(bytes=n * case["bits"] / 8 + 4 * -(-n // case["block"])
                    + case["vecs"] * (case["cols"] * x + case["rows"] * y)
                    + (case["rows"] * x if case["bias"] else 0), flops=2.0 * n * case["vecs"])
    total = case["total"]
    g = 4 if case["grad"] == "f32" else 2
    if case["op"] == "norm":
        return dict(bytes=total * g + 8, flops=2.0 * total)
    states = 16.0 if case["state"] == 32 else 4.0 + 16.0 / STATE_BLOCK
    w = 0 if case["weight"] == "none" else 2
    return dict(bytes=total * (8 + g + states + w), flops=total * (20.0 if case["state"] == 32 else 50.0))


# ------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "matvec":
        rows, cols, block = case["rows"], case["cols"], case["block"]
        n = rows * cols
        raw = s["codes"].to(torch.int64)
        if case["bits"] == 4:
            raw = torch.stack([raw % 16, raw // 16], 1).flatten()[:n]
        half = 2 ** (case["bits"] - 1)
        signed = raw - 2 * half * (raw >= half)
        w = signed.double()
        del raw, signed
        w *= s["scales"].double().repeat_interleave(block)[:n]
        y = s["x"].double() @ w.view(rows, cols).T
        return y if s["bias"] is None else y + s["bias"].double()
    g = s["g"].double()
    total = g.pow(2).sum().sqrt()
    clip = min(1.0, s["max_norm"] / float(total))
    norm = torch.tensor([float(total), clip], dtype=torch.float64, device="cuda")
    if case["op"] == "norm":
        return norm
    if case["clip"]:
        g *= clip
    t = STEP0 + 1
    eight = case["state"] == 8
    if eight:
        m = s["m"].double() * s["ms"].double().repeat_interleave(STATE_BLOCK)
        v = (s["v"].double() * s["vs"].double().repeat_interleave(STATE_BLOCK)).pow(2)
    else:
        m, v = s["m"].double(), s["v"].double()
    m = torch.lerp(g, m, BETA1)
    v = torch.lerp(g.pow(2), v, BETA2)
    del g
    update = m / (1 - BETA1 ** t) / ((v / (1 - BETA2 ** t)).sqrt() + EPS)
    p = s["p"].double() * (1 - LR * DECAY) - LR * update
    del update
    out = dict(p=p)
    if s["w"] is not None:
        out["w"] = p
    if case["clip"]:
        out["norm"] = norm
    if not eight:
        out.update(m=m, v=v)
        return out
    del s

    def grid(x, u, keep):
        """The e4m3 value reached from x / scale by floor(|x| / h + u) h, h the spacing there."""
        scale = x.view(-1, STATE_BLOCK).abs().amax(1) / 448
        y = x / scale.clamp(min=1e-300).repeat_interleave(STATE_BLOCK)
        size = y.abs()
        h = torch.exp2(torch.floor(torch.log2(size.clamp(min=2.0 ** -6))) - 3)
        k = torch.floor(size / h + u) * h
        if keep:
            k = torch.where(size > 0, k.clamp(min=2.0 ** -9), k)
        return torch.copysign(k.clamp(max=448), y), scale

    u = _random_bits(m.numel(), t)
    out["m"], out["ms"] = grid(m, ((u % 65536).double() + 0.5) / 65536, False)
    out["v"], out["vs"] = grid(v.sqrt(), ((u // 65536).double() + 0.5) / 65536, True)
    return out
