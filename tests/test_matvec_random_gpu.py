"""Products of random shapes, strides, types and numbers of vectors, exact as in test_matvec_gpu:
scales that are powers of two and small integers, so that any order of the sums gives equal bits."""
import random

import pytest
import torch
from test_matvec_gpu import DEV, gen, random_codes, weights

import quantized_zero_communication_gb300 as zpp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", range(8))
def test_random_products(seed):
    r = random.Random(seed)
    for case in range(100):
        rows, cols = int(2 ** r.uniform(0, 12)), int(2 ** r.uniform(0, 13))
        bits, block = r.choice((4, 8)), r.choice((64, 128, 256, 512, 1024, 2048, 4096))
        unit = r.choice((1, 4, 8, 128, block))  # any width, words, segments, blocks
        cols = max(unit, cols // unit * unit)
        vecs, n = r.choice((1, 1, 2, 3, 4, 5, 7, 8, 9, 12, 13, 16, 17, 20)), rows * cols
        dtype, g = r.choice((torch.float16, torch.bfloat16)), gen(1000 * seed + case)
        codes = random_codes(n, bits, g)
        scales = torch.exp2(torch.randint(-1, 2, (-(-n // block),), generator=g, device=DEV).float())
        top = max(1, min(3, 2 ** 21 // (cols * 2 ** (bits - 1) * 2)))
        stride = cols + r.choice((0, 0, 1, 3, 8))
        x = torch.randint(-top, top + 1, (vecs, stride), generator=g, device=DEV).to(dtype)[:, :cols]
        bias = torch.randint(-64, 65, (rows,), generator=g, device=DEV).to(dtype) if r.random() < 0.3 else None
        y = torch.full((vecs, rows + 5), 7.0, device=DEV)[:, :rows] if r.random() < 0.3 else None
        got = zpp.matvec_blockwise(codes, scales, x, rows, block, bits, bias=bias, dtype=torch.float32, y=y)
        want = x.double() @ weights(codes, scales, rows, cols, block, bits).T
        if bias is not None:
            want = want + bias.double()
        assert torch.equal(got.double(), want), (rows, cols, block, bits, vecs, dtype, stride)
