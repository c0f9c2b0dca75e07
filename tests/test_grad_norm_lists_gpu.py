"""The gradient norm over longer lists: both tables a launch's list may travel in (up to 16
tensors, and more), empty tensors anywhere, more chunks than the 64 places at which a launch writes
down a chunk's tensor, 16-byte alignment. Against 64 bits; the bound is that of fp32 partial sums
of at most 16384 squares, (64 + 10 + 2) 2^-24 of the sum and half of it for the root: 1e-5 is more than
twice that."""
import math
import random

import pytest
import torch

import quantized_zero_communication_gb300 as zpp

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def cut(sizes, dtype, seed, shift=0):
    """Tensors one after the other in a buffer, each at a multiple of 32 bytes (+ shift), NaN
    between them."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    per = 32 // dtype.itemsize
    skip = shift // dtype.itemsize
    at, end = [], skip
    for n in sizes:
        at.append(end)
        end += -(-n // per) * per
    flat = torch.full((end + per,), float("nan"), device=DEV, dtype=dtype)
    out = [flat[o:o + n] for o, n in zip(at, sizes)]
    # another magnitude in every tensor, so that one that is missed or read twice shows
    for i, t in enumerate(out):
        t.copy_(torch.randn(t.numel(), generator=gen, device=DEV) * (0.5 + i % 7))
    return out


def check(grads, max_norm=None):
    want = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    norm, coef = zpp.grad_norm(grads, max_norm=max_norm, pre_scale=0.5).tolist()
    assert abs(norm - 0.5 * want) <= 1e-5 * want
    clip = 1.0 if max_norm is None or want == 0 else min(1.0, max_norm / (0.5 * want))
    assert abs(coef - 0.5 * clip) <= 1e-5


def odd_sizes(count, seed, top):
    rng = random.Random(seed)
    return [rng.choice((1, 7, 8, 255, 4099, 16384, 16385, top)) for _ in range(count)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("count", [15, 16, 17, 150, 1023, 1024])
@pytest.mark.parametrize("shift", [0, 16])
def test_unequal_sizes(dtype, count, shift):
    grads = cut(odd_sizes(count, count, 100_003), dtype, count, shift)
    check(grads)
    check(grads, max_norm=1.0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("count", [12, 40, 1024])
@pytest.mark.parametrize("place", ["front", "middle", "end", "all but one"])
def test_runs_of_empty_tensors(dtype, count, place):
    sizes = odd_sizes(count, count, 300_001)
    third = count // 3
    lo, hi = dict([("front", (0, third)), ("middle", (third, 2 * third)), ("end", (2 * third, count)),
                   ("all but one", (0, count - 1))])[place]
    for i in range(lo, hi):
        sizes[i] = 0
    check(cut(sizes, dtype, count))


def test_all_empty():
    check([torch.empty(0, device=DEV) for _ in range(20)])


@pytest.mark.parametrize("dtype", DTYPES)
def test_one_tensor_of_a_list_is_aligned_to_16_bytes_only(dtype):
    grads = cut([20_000] * 30, dtype, 3)
    grads[17] = cut([50_001], dtype, 4, shift=16)[0]
    check(grads)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("count, top", [(3, 40_000_003), (200, 1_000_003)])
def test_many_chunks(dtype, count, top):
    """Some thousands of chunks: 64 or more to a written place."""
    rng = random.Random(count)
    check(cut([rng.choice((top, top // 3, 5)) for _ in range(count)], dtype, 5))


@pytest.mark.parametrize("bits", [32, 8])
def test_clipped_step_over_more_tensors_than_a_launch_takes(bits):
    """Equals the norm's factor handed to the step, bit for bit."""
    sizes = [n % 3001 for n in odd_sizes(900, 9, 3000)]
    code = torch.float32 if bits == 32 else torch.float8_e4m3fn
    grads = cut(sizes, torch.bfloat16, 6)
    params = [torch.ones(n, device=DEV) for n in sizes]
    opt = zpp.AdamW(params, lr=1e-2, weight_decay=0.0, state_bits=bits, seed=4)
    norm = opt.step(grads, max_norm=2.0)
    total = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    assert abs(float(norm[0]) - total) <= 1e-5 * total
    plain = [torch.ones(n, device=DEV) for n in sizes]
    m, v = ([torch.zeros(n, device=DEV).to(code) for n in sizes] for _ in range(2))
    a, b = ([torch.zeros(-(-n // 256), device=DEV) for n in sizes] for _ in range(2))
    zpp.adamw_step(plain, grads, m, v, step=1, lr=1e-2, scales=None if bits == 32 else (a, b), seed=4,
                   grad_scale=norm[1:])
    for x, y in ((opt.params, plain), (opt.exp_avg, m), (opt.exp_avg_sq, v)):
        assert all(torch.equal(s.view(torch.uint8), t.view(torch.uint8)) for s, t in zip(x, y))
