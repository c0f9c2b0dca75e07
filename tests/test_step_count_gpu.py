"""The number of an AdamW step counts the steps that were taken: one that a non-finite factor
skipped leaves the bias corrections, the rounding bits and the saved count where they were. Runs
with skipped steps are compared bit for bit with runs without them."""
import math

import pytest
import torch

import quantized_zero_communication_gb300 as zpp

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
SIZES = (1000, 33, 70_001)
HP = dict(lr=3e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1)


def normal(n, sigma, seed):
    return torch.randn(n, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV) * sigma


def fresh(bits, step=0):
    params = [normal(n, 0.02, n) for n in SIZES]
    weights = [torch.zeros(n, device=DEV, dtype=torch.bfloat16) for n in SIZES]
    return zpp.AdamW(params, state_bits=bits, weights=weights, seed=3, step=step, **HP)


def grads(t, bad=None):
    out = [normal(n, 1.0, 1000 * t + n).half() for n in SIZES]
    if bad is not None:
        out[1][7] = bad
    return out


def everything(opt):
    lists = [opt.params, opt.exp_avg, opt.exp_avg_sq, opt.weights, *(opt.scales or ())]
    return [t.clone().view(torch.uint8) for ts in lists for t in ts]


def same(a, b):
    assert all(torch.equal(x, y) for x, y in zip(everything(a), everything(b), strict=True))
    assert a.steps == b.steps and a.state()["step"] == b.state()["step"]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_overflowed_clipped_steps_do_not_count(bits, bad):
    hurt, clean = fresh(bits), fresh(bits)
    for t in range(10):  # as while a loss scale is being found
        norm = hurt.step(grads(t, bad), max_norm=1.0, pre_scale=2.0 ** -10)
        assert math.isnan(float(norm[1])) and hurt.steps == 0
    for opt in (hurt, clean):
        opt.step(grads(20), max_norm=1.0)
    same(hurt, clean)
    assert clean.steps == 1
    hurt.step(grads(21, bad), max_norm=1.0)
    for opt in (hurt, clean):
        opt.step(grads(22), max_norm=1.0)
    same(hurt, clean)


@pytest.mark.parametrize("bits", [32, 8])
def test_steps_of_every_kind_share_the_count(bits):
    """Unscaled, clipped and outside-scaled steps in turn, skipped ones between them, from a
    resumed count; the clean run takes every step by the same call or, where the factor is one,
    by another."""
    one = torch.ones(1, device=DEV)
    hurt, clean = fresh(bits, step=5), fresh(bits, step=5)
    hurt.step(grads(1))
    clean.step(grads(1), grad_scale=one)
    hurt.step(grads(2), grad_scale=torch.full((1,), math.inf, device=DEV))
    hurt.step(grads(3))
    clean.step(grads(3))
    hurt.step(grads(4, math.nan), pre_scale=0.5)
    for opt in (hurt, clean):
        opt.step(grads(5), max_norm=0.5, pre_scale=0.25)
    hurt.step(grads(6))
    clean.step(grads(6), max_norm=math.inf)
    same(hurt, clean)
    assert hurt.steps == 9
    again = zpp.AdamW([p.clone() for p in hurt.params], weights=[w.clone() for w in hurt.weights],
                      **HP, **{k: [x.clone() for x in v] if k.startswith("exp") else
                               v and tuple([x.clone() for x in s] for s in v) if k == "scales" else v
                               for k, v in hurt.state().items()})
    for opt in (hurt, again):
        opt.step(grads(7))
    same(hurt, again)


@pytest.mark.parametrize("clip", [True, False])
def test_replayed_steps_count(clip):
    """A captured step, replayed, is the next step each time."""
    opt, want = fresh(8), fresh(8)
    static = grads(0)
    kw = dict(max_norm=1.0) if clip else {}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        opt.step(static, **kw)
    torch.cuda.current_stream().wait_stream(s)
    want.step(grads(0), **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step(static, **kw)
    for t in (1, 2, 3):
        g = grads(t, math.inf if clip and t == 2 else None)
        for a, b in zip(static, g):
            a.copy_(b)
        graph.replay()
        if not (clip and t == 2):
            want.step(g, **kw)
        same(opt, want)
    for o in (opt, want):
        o.step(grads(9))
    same(opt, want)


def test_a_refused_step_does_not_count():
    opt = fresh(32)
    opt.step(grads(1), max_norm=1.0)
    with pytest.raises(ValueError):
        opt.step(grads(2)[:2], max_norm=1.0)
    with pytest.raises(zpp.ZppError):  # 16-byte alignment
        opt.step([torch.zeros(n + 1, device=DEV, dtype=torch.float16)[1:] for n in SIZES], max_norm=1.0)
    with pytest.raises(zpp.ZppError):
        opt.step(grads(2), max_norm=-1.0)
    assert opt.steps == 1


def test_the_count_can_be_set():
    opt, want = fresh(8), fresh(8, step=41)
    opt.steps = 41
    for o in (opt, want):
        o.step(grads(1), max_norm=1.0)
    same(opt, want)
    assert opt.steps == 42
