"""Calls of the fp8 products and the Newton-Schulz steps at their edges: more than 2^31 elements, host
threads side by side, a first call inside a captured graph, inference mode, scales and vectors of
unusual form. Bounds as in test_fp8_gpu.py and test_muon_gpu.py."""
import subprocess
import sys
import threading

import pytest
import torch

import quantized_zero_communication_gb300 as zpp
from quantized_zero_communication_gb300 import build
from test_fp8_gpu import DEV, gen, integers, powers, product, spread
from test_muon_gpu import USUAL, matrix, norm

pytestmark = pytest.mark.gpu


def test_quantiser_beyond_32_bits():
    rows, cols = 70_000, 32_768  # 2.3e9 values
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    x[-3:] = torch.randn(3, cols, generator=gen(1), device=DEV).bfloat16()
    codes, scales, codes_t, scales_t = zpp.quant_fp8(x, 1, transposed=True)
    want = zpp.quant_fp8(x[-3:])
    assert torch.equal(codes[-3:].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(scales[-3:], want[1])
    assert not codes[:-3].view(torch.uint8).any() and not scales[:-3].any()
    last = x[rows // 128 * 128:].t().contiguous()
    want = zpp.quant_fp8(last)
    assert torch.equal(codes_t[:, rows // 128 * 128:].reshape(last.shape).view(torch.uint8), want[0].view(torch.uint8))
    assert torch.equal(scales_t[:, -1:], want[1]) and not scales_t[:, :-1].any()


def test_product_beyond_32_bits():
    m, n, k = 70_000, 40_000, 16  # 2.8e9 results
    a, b = integers(m, k, 1), integers(n, k, 2)
    sa, sb = powers(m, k, 1, 3), powers(n, k, 128, 4)
    y = zpp.matmul_fp8(a, sa, b, sb)
    for rows in (slice(0, 40), slice(m - 40, m)):
        want, _ = product(a[rows], sa[rows], 1, b, sb, 128)
        assert torch.equal(y[rows], want.bfloat16())
    del y
    # codes beyond 4 GB, read by few rows
    n, k = 140_000, 32_768
    b = torch.zeros(n, k, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    b[-200:] = integers(200, k, 5)
    a, sb = integers(2, k, 6), powers(n, k, 1, 7)
    y = zpp.matmul_fp8(a, powers(2, k, 1, 8), b, sb, dtype=torch.float32)
    want, size = product(a, powers(2, k, 1, 8), 1, b[-200:], sb[-200:], 1)
    assert ((y[:, -200:].double() - want).abs() <= 2.0 ** -24 * (20 + k / 128) * size).all()
    assert not y[:, :-200].any()


def test_steps_beyond_32_bits():
    """X^T X of the whole in 64 bits by parts; the result's first and last rows are X's times a polynomial."""
    rows, cols = (1 << 22) + 5, 600
    x = torch.randn(rows, cols, generator=gen(3), device=DEV, dtype=torch.float16)
    got = zpp.orthogonalize(x)
    gram = torch.zeros(cols, cols, dtype=torch.float64, device=DEV)
    for at in range(0, rows, 1 << 19):
        part = x[at:at + (1 << 19)].double()
        gram += part.t() @ part
    gram /= torch.trace(gram)
    total = torch.eye(cols, dtype=torch.float64, device=DEV)
    size = sum(float(x[at:at + (1 << 19)].double().square().sum()) for at in range(0, rows, 1 << 19)) ** 0.5
    for _ in range(5):
        a, b, c = USUAL
        step = a * torch.eye(cols, dtype=torch.float64, device=DEV) + b * gram + c * gram @ gram
        total, gram = total @ step, gram @ step @ step
    for part in (slice(0, 1000), slice(rows - 1000, rows)):
        want = x[part].double() / size @ total
        # fp16 of 2^-11 elements: half a step of 2^-24 at most, 2^-11 of larger ones, and the steps' 1e-3
        assert norm(got[part].double() - want) <= (2.0 ** -11 + 2e-3) * norm(want) + want.numel() ** 0.5 * 2.0 ** -25


def test_host_threads():
    """Four threads, each on a stream of its own, through products and steps of their own sizes."""
    jobs = []
    for i in range(4):
        m, n, k = 30 + 60 * i, 200 + 100 * i, 500 + 300 * i
        a, b = integers(m, k, i), integers(n, k, i + 10)
        sa, sb = powers(m, k, 1, i), powers(n, k, 128, i)
        x = matrix(100 + 60 * i, 150, i).bfloat16()
        jobs.append((a, sa, b, sb, x, product(a, sa, 1, b, sb, 128)[0], zpp.orthogonalize(x)))
    torch.cuda.synchronize()
    bad = []

    def work(a, sa, b, sb, x, want, flat):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                y = zpp.matmul_fp8(a, sa, b, sb, dtype=torch.float32)
                z = zpp.orthogonalize(x)
            torch.cuda.current_stream().synchronize()
            if not (torch.equal(y.double(), want) and torch.equal(z, flat)):
                bad.append(x.shape)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and zpp.zpp_device_fault() == 0


def test_first_call_in_a_captured_graph():
    code = """
import torch, quantized_zero_communication_gb300 as zpp
x = torch.randn(200, 300, device="cuda").bfloat16()
w = torch.randn(260, 300, device="cuda")
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    y = zpp.matmul_fp8(*zpp.quant_fp8(x), *zpp.quant_fp8(w, 128))
    z = zpp.orthogonalize(x)
graph.replay()
torch.cuda.synchronize()
assert torch.equal(y, zpp.matmul_fp8(*zpp.quant_fp8(x), *zpp.quant_fp8(w, 128)))
assert torch.equal(z, zpp.orthogonalize(x))
"""
    done = subprocess.run([sys.executable, "-c", code], cwd=build.ROOT, capture_output=True, text=True)
    assert done.returncode == 0, done.stderr[-2000:]


def test_unusual_forms():
    a, b = integers(40, 700, 1), integers(50, 700, 2)
    one = torch.exp2(torch.arange(40, device=DEV).float() % 5)[:, None]
    sa, sb = one.expand(40, 6), torch.ones(1, 1, device=DEV).expand(1, 6)  # a scale a row; one for all
    want, _ = product(a, sa, 1, b, sb, 128)
    assert torch.equal(zpp.matmul_fp8(a, sa, b, sb, dtype=torch.float32).double(), want)
    wide = powers(80, 700 * 2, 1, 3)
    sa = wide[::2, ::2][:, :6]  # every other one
    want, _ = product(a, sa, 1, b, sb, 128)
    assert torch.equal(zpp.matmul_fp8(a, sa, b, sb, dtype=torch.float32).double(), want)
    x = torch.randn(300, generator=gen(4), device=DEV).bfloat16()  # a vector
    w = torch.randn(70, 300, generator=gen(5), device=DEV)
    y = zpp.linear_fp8(x, w)
    assert y.shape == (70,) and torch.equal(y, zpp.linear_fp8(x[None], w)[0])
    with torch.inference_mode():
        t = torch.randn(5, 300, device=DEV).bfloat16()
        out = zpp.linear_fp8(t, w)
        codes = zpp.quant_fp8(t)
        zpp.quant_fp8(t, out=codes)
        zpp.matmul_fp8(*codes, *zpp.quant_fp8(w, 128), y=out)
        assert torch.equal(out, zpp.linear_fp8(t, w))
    assert zpp.Muon([torch.zeros(0, 5, device=DEV)]).step([torch.zeros(0, 5, device=DEV)]) is None
    value = codes[0].to(torch.float64) * spread(codes[1], 1, 5, 300)
    assert ((value - t.double()).abs() <= 2.0 ** -4 * t.double().abs() + codes[1].double().max() * 2.0 ** -10).all()
