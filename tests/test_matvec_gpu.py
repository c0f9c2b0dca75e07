"""The product with block-quantised weights against its definition in 64 bits.

Two kinds of check. Exact: scales that are powers of two and small integer inputs make every
product and partial sum an integer multiple of a power of two that fp32 holds, whatever the
order, so the result has to be equal. Rounded: real data within
  |dy| <= 2u (cols / 16 + 32) sum |w x| + half an ulp of the output type,  u = 2^-24,
which allows every 16-element step of a running sum an error of 2u of the largest partial sum,
and the joins and the scale's products 32 more."""
import pytest
import torch

import quantized_zero_communication_gb300 as zpp

pytestmark = pytest.mark.gpu

DEV, U = "cuda:0", 2.0 ** -24
HALF_ULP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def unpack(codes, n, bits):
    c = codes.view(torch.int8)
    if bits == 4:
        c = torch.stack([(c << 4) >> 4, c >> 4], 1).view(-1)
    return c[:n].double()


def weights(codes, scales, rows, cols, block, bits):
    q = unpack(codes, rows * cols, bits)
    return (q * scales.double().repeat_interleave(block)[:rows * cols]).view(rows, cols)


def random_codes(n, bits, g):
    top = 2 ** (bits - 1) - 1
    q = torch.randint(-top, top + 1, (n,), generator=g, device=DEV).to(torch.int8)
    if bits == 4:
        q = torch.cat([q, q.new_zeros(n % 2)])
        q = (q[0::2] & 15) | (q[1::2] << 4)
    return q.view(torch.uint8)


def check_exact(rows, cols, block, bits, vecs, dtype, seed=0, bias=False, out=torch.float32):
    g = gen(seed)
    n = rows * cols
    codes = random_codes(n, bits, g)
    scales = torch.exp2(torch.randint(-1, 2, (-(-n // block),), generator=g, device=DEV).float())
    # |sum| stays below 2^23 halves: at most cols * qmax * 2 * top
    top = max(1, min(3, 2 ** 21 // (cols * (2 ** (bits - 1)) * 2)))
    x = torch.randint(-top, top + 1, (vecs, cols), generator=g, device=DEV).to(dtype)
    b = torch.randint(-64, 65, (rows,), generator=g, device=DEV).to(dtype) if bias else None
    y = zpp.matvec_blockwise(codes, scales, x, rows, block, bits, bias=b, dtype=out)
    want = x.double() @ weights(codes, scales, rows, cols, block, bits).T
    if bias:
        want = want + b.double()
    assert y.shape == (vecs, rows)
    assert torch.equal(y, want.float().to(out))


@pytest.mark.parametrize("block", [64, 128, 256, 512, 1024, 2048, 4096])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("vecs", [1, 3])
def test_whole_blocks_per_row(block, bits, vecs):
    for rows, k in ((1, 1), (17, 1), (100, 3), (33, 2)):
        check_exact(rows, block * k, block, bits, vecs, torch.float16, seed=rows)


@pytest.mark.parametrize("cols", [1, 2, 7, 8, 9, 31, 63, 64, 65, 100, 127, 192, 255, 1000, 1003, 4097])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("block", [64, 4096])
def test_any_width(cols, bits, block):
    """Widths that are not whole blocks: rows start inside a block, a byte, a word."""
    for rows, vecs in ((1, 1), (3, 2), (65, 5)):
        check_exact(rows, cols, block, bits, vecs, torch.bfloat16, seed=cols)


@pytest.mark.parametrize("vecs", [1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 31, 32, 33, 40, 70])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_numbers_of_vectors(vecs, bits, dtype):
    check_exact(130, 512, 64, bits, vecs, dtype, seed=vecs, bias=True)
    check_exact(50, 1536, 256, bits, vecs, dtype, seed=vecs)
    check_exact(21, 203, 128, bits, vecs, dtype, seed=vecs, bias=True)


@pytest.mark.parametrize("rows,cols,block", [(4096, 8192, 128), (16, 65536, 2048), (1, 131072, 64),
                                             (30000, 512, 512), (257, 14336, 64), (12, 200_003, 64)])
@pytest.mark.parametrize("bits", [4, 8])
def test_long_and_tall(rows, cols, block, bits):
    check_exact(rows, cols, block, bits, 1, torch.float16)
    check_exact(rows, cols, block, bits, 9, torch.bfloat16)


@pytest.mark.parametrize("rows,cols,vecs", [
    (3, 100_001, 5),    # x over a whole cluster's shared memory
    (2, 300_001, 8),    # and a few vectors at a time
    (2, 800_003, 2)])   # and beyond it
@pytest.mark.parametrize("bits", [4, 8])
def test_very_long_rows(rows, cols, vecs, bits):
    check_exact(rows, cols, 128, bits, vecs, torch.float16, bias=True)


@pytest.mark.parametrize("rows", [1, 15, 31, 32, 33, 511, 512, 513, 2500])
@pytest.mark.parametrize("bits", [4, 8])
def test_odd_width_row_counts(rows, bits):
    """Rows are gathered by the place of their first code in a 16-byte chunk."""
    for cols in (5, 333, 1001):
        check_exact(rows, cols, 64, bits, 2, torch.float16, seed=rows)


@pytest.mark.parametrize("rows,cols,block,bits,vecs,dtype,out", [
    (1000, 4096, 128, 4, 1, torch.bfloat16, torch.bfloat16),
    (1000, 4096, 64, 4, 8, torch.float16, torch.float32),
    (513, 8192, 2048, 8, 1, torch.float16, torch.float16),
    (513, 8192, 256, 8, 12, torch.bfloat16, torch.float32),
    (2001, 1003, 64, 4, 3, torch.float16, torch.float32),
    (100, 30001, 512, 8, 2, torch.bfloat16, torch.float16)])
def test_real_weights(rows, cols, block, bits, vecs, dtype, out):
    """Weights through the library's own quantiser."""
    g = gen(rows)
    w = (torch.randn(rows * cols, generator=g, device=DEV) * 0.02).to(dtype)
    codes, scales = zpp.quant_blockwise(w, block, bits)
    x = torch.randn(vecs, cols, generator=g, device=DEV).to(dtype)
    b = torch.randn(rows, generator=g, device=DEV).to(dtype)
    y = zpp.matvec_blockwise(codes, scales, x, rows, block, bits, bias=b, dtype=out)
    W = weights(codes, scales, rows, cols, block, bits)
    want = x.double() @ W.T + b.double()
    mass = x.double().abs() @ W.abs().T + b.double().abs()
    tol = 2 * U * (cols / 16 + 32) * mass + HALF_ULP[out] * want.abs() * (1 + 1e-3) + 2.0 ** -25
    bad = (y.double() - want).abs() > tol
    assert not bool(bad.any()), float(((y.double() - want).abs() / tol).max())
    again = zpp.matvec_blockwise(codes, scales, x, rows, block, bits, bias=b, dtype=out)
    assert torch.equal(y, again)


@pytest.mark.parametrize("cols,block", [(256, 64), (203, 64)])
def test_strides_shapes_and_buffers(cols, block):
    """Row strides of x and y (odd ones too), leading dimensions, a given output, guards."""
    g, rows = gen(5), 45
    codes = random_codes(rows * cols, 4, g)
    scales = torch.ones(-(-rows * cols // block), device=DEV)
    W = weights(codes, scales, rows, cols, block, 4)
    for pad in (0, 1, 8):
        wide = torch.randint(-3, 4, (6, cols + pad), generator=g, device=DEV).to(torch.bfloat16)
        wide[:, cols:] = float("nan")  # outside the rows: never read into a result
        x = wide[:, :cols]
        buf = torch.full((6, rows + pad), 9.0, device=DEV)
        y = zpp.matvec_blockwise(codes, scales, x, rows, block, 4, y=buf[:, :rows])
        assert torch.equal(y, (x.double() @ W.T).float()) and y.data_ptr() == buf.data_ptr()
        assert bool((buf[:, rows:] == 9).all())
    x = torch.randint(-3, 4, (2, 3, cols), generator=g, device=DEV).half()
    y = zpp.matvec_blockwise(codes, scales, x, rows, block, 4)
    assert y.shape == (2, 3, rows) and y.dtype == torch.float16
    assert torch.equal(y, (x.double() @ W.T).half())
    v = zpp.matvec_blockwise(codes, scales, x[0, 0], rows, block, 4)
    assert v.shape == (rows,) and torch.equal(v, y[0, 0])
    assert zpp.matvec_blockwise(codes, scales, x[:, :0], rows, block, 4).shape == (2, 0, rows)
    empty = zpp.matvec_blockwise(codes[:0], scales[:0], x, 0, block, 4)
    assert empty.shape == (2, 3, 0)


def test_infinite_and_nan_inputs_reach_only_their_vector():
    rows, cols, block = 33, 512, 128
    g = gen(6)
    codes = random_codes(rows * cols, 4, g)
    scales = torch.ones(rows * cols // block, device=DEV)
    x = torch.randint(-3, 4, (9, cols), generator=g, device=DEV).half()
    clean = zpp.matvec_blockwise(codes, scales, x, rows, block, 4, dtype=torch.float32)
    x[4, 77], x[8, 3] = float("nan"), float("inf")
    y = zpp.matvec_blockwise(codes, scales, x, rows, block, 4, dtype=torch.float32)
    others = [0, 1, 2, 3, 5, 6, 7]
    assert torch.equal(y[others], clean[others])
    assert bool(torch.isnan(y[4]).all()) and not bool(torch.isfinite(y[8]).any())


def test_infinite_scale_of_a_neighbouring_row_stays_out():
    """A row ends inside a word and a block: the other row's part does not reach it."""
    rows, cols, block = 2, 67, 64
    codes = torch.full(((rows * cols + 1) // 2,), 0x11, dtype=torch.uint8, device=DEV)
    scales = torch.tensor([1.0, 1.0, float("inf")], device=DEV)  # elements 128 .. 133: row 1
    y = zpp.matvec_blockwise(codes, scales, torch.ones(cols, device=DEV).half(), rows, block, 4)
    assert float(y[0]) == 67.0 and float(y[1]) == float("inf")


def test_another_stream():
    g = gen(7)
    codes = random_codes(512 * 1024, 4, g)
    scales = torch.ones(512 * 1024 // 64, device=DEV)
    x = torch.randint(-3, 4, (1, 1024), generator=g, device=DEV).half()
    want = zpp.matvec_blockwise(codes, scales, x, 512, 64, 4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = zpp.matvec_blockwise(codes, scales, x, 512, 64, 4)
    s.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("cols", [8192, 8191])
def test_offsets_beyond_32_bits(cols):
    """Code bytes and element numbers past 2^32: the first and the last rows of 4.9 GB."""
    g, rows, block = gen(8), 600_000, 4096
    n = rows * cols
    codes = torch.randint(0, 256, (n,), generator=g, device=DEV, dtype=torch.uint8)
    codes[codes == 128] = 0  # -128 is no code
    scales = torch.exp2(torch.randint(-1, 2, (-(-n // block),), generator=g, device=DEV).float())
    x = torch.randint(-1, 2, (2, cols), generator=g, device=DEV).half()
    y = zpp.matvec_blockwise(codes, scales, x, rows, block, 8, dtype=torch.float32)
    for lo in (0, rows - 64):
        part = slice(lo * cols, (lo + 64) * cols)
        at = torch.arange(part.start, part.stop, device=DEV) // block
        w = (codes[part].view(torch.int8).double() * scales[at].double()).view(64, cols)
        assert torch.equal(y[:, lo:lo + 64], (x.double() @ w.T).float())


def test_in_a_cuda_graph():
    """Captured calls (overlapped launches among them) replay on new inputs."""
    g, rows, cols = gen(9), 320, 1024
    w = torch.randn(rows * cols, generator=g, device=DEV).half()
    codes, scales = zpp.quant_blockwise(w, 128, 4)
    x = torch.randn(1, cols, generator=g, device=DEV).half()
    a, b = torch.empty(1, rows, device=DEV).half(), torch.empty(1, rows, device=DEV).half()

    def work():
        zpp.matvec_blockwise(codes, scales, x, rows, 128, 4, y=a)
        zpp.matvec_blockwise(codes, scales, x[:, :], rows, 128, 4, y=b)
        b.add_(a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for seed in (1, 2):
        x.copy_(torch.randn(1, cols, generator=gen(seed), device=DEV))
        graph.replay()
        want = zpp.matvec_blockwise(codes, scales, x, rows, 128, 4)
        assert torch.equal(a, want) and torch.equal(b, want + want)


def test_chains_of_calls_see_each_others_results():
    """Each call's input is the output of the one before, back to back on one stream: an
    overlapped launch must not read it early."""
    g, d = gen(10), 512
    mats = [zpp.quant_blockwise(torch.randn(d * d, generator=g, device=DEV).half() / d ** 0.5, 128, 4)
            for _ in range(4)]
    x = torch.randn(1, d, generator=g, device=DEV).half()
    want = x
    for codes, scales in mats * 8:
        want = zpp.matvec_blockwise(codes, scales, want, d, 128, 4)
        torch.cuda.synchronize()
    for _ in range(20):
        got = x
        for codes, scales in mats * 8:
            got = zpp.matvec_blockwise(codes, scales, got, d, 128, 4)
        assert torch.equal(got, want)


@pytest.mark.parametrize("vecs", [1, 2, 3, 5])
@pytest.mark.parametrize("bits, block, segments", [(4, 64, 3), (4, 128, 5), (4, 128, 11), (8, 64, 5)])
def test_infinite_scale_of_a_rows_last_block_gives_infinity(bits, block, segments, vecs):
    # rows of fewer segments than a warp takes at a time, or of a part more
    cols, rows = segments * (128 if bits == 4 else 64), 40
    n = rows * cols
    codes = torch.full((n * bits // 8,), 0x11 if bits == 4 else 1, dtype=torch.uint8, device=DEV)
    scales = torch.ones(rows, cols // block, device=DEV)
    scales[7, -1] = scales[20, -1] = float("inf")
    x = torch.ones(vecs, cols, device=DEV, dtype=torch.bfloat16)
    y = zpp.matvec_blockwise(codes, scales.view(-1), x, rows, block, bits, dtype=torch.float32)
    want = torch.full((vecs, rows), float(cols), device=DEV)
    want[:, 7] = want[:, 20] = float("inf")
    assert torch.equal(y, want)


@pytest.mark.parametrize("rows, cols", [(1, 8), (3, 24), (33, 40), (1027, 136), (515, 1032), (64, 8200),
                                        (2, 800_008)])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("vecs", [1, 8, 13])
def test_exact_rows_that_start_at_words(rows, cols, bits, vecs):
    check_exact(rows, cols, 64, bits, vecs, torch.bfloat16, seed=rows + vecs)
    check_exact(rows, cols - cols % 8 + 4, 2048, bits, vecs, torch.float16, seed=rows + vecs, bias=True)


def test_words_with_strides_of_x():
    """The width allows whole words, the stride of x does or does not."""
    rows, cols, g = 100, 1000, gen(21)
    codes = random_codes(rows * cols, 4, g)
    scales = torch.exp2(torch.randint(-1, 2, (-(-rows * cols // 128),), generator=g, device=DEV).float())
    want = weights(codes, scales, rows, cols, 128, 4)
    for stride in (1000, 1001, 1004, 1008):
        x = torch.randint(-3, 4, (5, stride), generator=g, device=DEV).half()[:, :cols]
        y = zpp.matvec_blockwise(codes, scales, x, rows, 128, 4, dtype=torch.float32)
        assert torch.equal(y.double(), x.double() @ want.T)


def test_stale_shared_memory_stays_out():
    """Chunks past a row's end meet what an earlier call left in shared memory: infinite scales."""
    g = gen(22)
    big = 4096 * 1000
    codes = random_codes(big, 4, g)
    x = torch.ones(3, 1000, device=DEV).half()
    zpp.matvec_blockwise(codes, torch.full((big // 64,), float("inf"), device=DEV), x, 4096, 64, 4)
    for cols in (40, 72, 1000, 1003):
        check_exact(600, cols, 64, 4, 3, torch.float16, seed=cols)


@pytest.mark.parametrize("rows, cols", [(5, 128), (70, 384), (600, 1280), (33, 8320)])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("block", [64, 256, 512, 2048, 4096])
def test_exact_whole_segments_in_blocks_across_rows(rows, cols, bits, block):
    for vecs in (1, 2, 3, 8, 17):
        check_exact(rows, cols, block, bits, vecs, torch.bfloat16, seed=rows + vecs)
