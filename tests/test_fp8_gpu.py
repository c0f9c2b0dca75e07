"""The e4m3 quantiser and the products of e4m3 matrices against their definitions in 64 bits.

Quantiser: every code and scale has to be equal. Products, two kinds of check. Exact: codes that
are small integers and scales that are powers of two make every product and partial sum an integer
multiple of a power of two that fp32 holds, so the result has to be equal. Rounded: real data within
  |dy| <= (20 + K / 128) u S + half an ulp of the output type,  u = 2^-24, S = sum |a b| of the values:
a block's sum takes four steps of the matrix unit, each off by at most 4u of its terms' magnitudes
(aligned to the largest and cut), the scales' product and its use 4u, and the running sum u a block."""
import pytest
import torch

import quantized_zero_communication_gb300 as zpp

pytestmark = pytest.mark.gpu

DEV, U = "cuda:0", 2.0 ** -24
HALF_ULP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
E4M3 = torch.float8_e4m3fn
TYPES = (torch.float16, torch.bfloat16, torch.float32)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def spread(scales, tile, rows, cols):
    """A scale for every element."""
    ones = torch.ones(tile, 128, dtype=torch.float64, device=DEV)
    return torch.kron(scales.double().contiguous(), ones)[:rows, :cols]


def pow2(e):
    """2^e from its bits (torch.ldexp's powers are off by an ulp in 64 bits)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def grid(x, tile):
    """(code values, scales) of the definition."""
    x = x.double()
    rows, cols = x.shape
    finite = torch.where(x.isfinite(), x.abs(), 0.0)
    down, across = -(-rows // tile), -(-cols // 128)
    wide = torch.zeros(down * tile, across * 128, dtype=torch.float64, device=DEV)
    wide[:rows, :cols] = finite
    top = wide.view(down, tile, across, 128).amax((1, 3))
    part, power = torch.frexp(top)  # 448 = 7/8 * 2^9
    power = (power - torch.where(part <= 0.875, 9, 8)).clamp(min=-126)
    scales = torch.where(top > 0, pow2(power), 0.0)
    full = spread(scales, tile, rows, cols)
    v = torch.where(full > 0, x / full, x * 0.0)
    part, power = torch.frexp(v)
    h = pow2(power.clamp(min=-5) - 4)  # spacing: 3 bits after the first
    v = torch.round(v / h) * h
    return torch.where(x.isfinite(), v, torch.nan), scales


def check_quant(x, tile, out):
    want, scales = grid(x, tile)
    assert torch.equal(out[1].double(), scales)
    got = out[0].to(torch.float64)
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(), want.nan_to_num())
    assert out[0].stride(-2) % 16 == 0 or out[0].shape[-2] <= 1
    if len(out) == 4:
        want, scales = grid(x.t(), tile)
        assert torch.equal(out[3].double(), scales)
        got = out[2].to(torch.float64)
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got.nan_to_num(), want.nan_to_num())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tile", (1, 128))
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 16), (5, 100), (128, 128), (127, 129),
                                       (130, 257), (300, 1003), (1, 5000), (1000, 1), (129, 512)])
def test_quantiser_equals_its_definition(rows, cols, tile, dtype):
    g = gen(rows * 7 + cols)
    x = torch.randn(rows, cols, generator=g, device=DEV)
    x = (x * torch.exp(3 * torch.randn(rows, 1, generator=g, device=DEV))).to(dtype)
    for transposed in (False, True):
        check_quant(x, tile, zpp.quant_fp8(x, tile, transposed=transposed))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tile", (1, 128))
def test_quantiser_borders(tile, dtype):
    """Zeros, the largest and smallest values, ties between codes, amax on and next to 448 * 2^e."""
    x = torch.zeros(260, 384, device=DEV, dtype=dtype)
    info = torch.finfo(dtype)
    x[0, :4] = torch.tensor([info.max, -info.max, info.tiny, 0.0], dtype=dtype)
    x[1, 128:130] = torch.tensor([info.smallest_normal / 2 ** 3, -info.smallest_normal], dtype=dtype)
    for i, top in enumerate((448.0, 449.0, 447.0, 450.0, 224.0, 225.0, 1.75, 1.7578125)):
        x[3 + i, 0] = top
        x[3 + i, 1:100] = torch.arange(99, device=DEV).to(dtype) * (top / 256)
    steps = torch.arange(128, device=DEV).double()
    x[20, :128] = (steps / 16).to(dtype)        # every tie of the spacing 1/8 .. 1
    x[21, :128] = (steps * 2.0 ** -11).to(dtype)  # among the subnormal codes
    x[21, 0] = 448.0
    x[140, 200] = -3.0
    check_quant(x, tile, zpp.quant_fp8(x, tile, transposed=True))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tile", (1, 128))
def test_quantiser_passes_over_values_that_are_not_finite(tile, dtype):
    x = torch.randn(200, 300, generator=gen(0), device=DEV).to(dtype)
    x[3, 5], x[3, 140], x[150, 299], x[0, 0] = float("inf"), float("nan"), float("-inf"), float("nan")
    x[7] = float("nan")
    x[8] = float("inf")
    check_quant(x, tile, zpp.quant_fp8(x, tile, transposed=True))


@pytest.mark.parametrize("dtype", TYPES)
def test_quantiser_strides_shapes_and_buffers(dtype):
    base = torch.randn(70, 400, generator=gen(1), device=DEV).to(dtype)
    for x in (base[:, :300], base[:, 1:301], base[3:40, 7:136], base[5:6, 3:9]):
        check_quant(x, 1, zpp.quant_fp8(x, 1, transposed=True))
        check_quant(x, 128, zpp.quant_fp8(x, 128, transposed=True))
    x = base[:, :390].contiguous().view(7, 10, 390)
    codes, scales = zpp.quant_fp8(x)
    assert codes.shape == x.shape and scales.shape == (70, 4)
    check_quant(x.view(70, 390), 1, (codes.reshape(70, 390), scales))
    # buffers of the caller: what lies between the rows stays as it was
    codes = torch.full((70, 416), 0x55, dtype=torch.uint8, device=DEV)
    back = torch.full((390, 96), 0x55, dtype=torch.uint8, device=DEV)
    out = (codes.view(E4M3)[:, :390], torch.empty(70, 4, device=DEV), back.view(E4M3)[:, :70],
           torch.empty(390, 1, device=DEV))
    got = zpp.quant_fp8(base[:, :390], 1, transposed=True, out=out)
    assert all(a is b for a, b in zip(got, out))
    check_quant(base[:, :390], 1, got)
    assert (codes[:, 390:] == 0x55).all() and (back[:, 70:] == 0x55).all()
    assert zpp.quant_fp8(base[:0])[0].shape == (0, 400)


def test_quantiser_of_more_row_tiles_than_a_grid_holds():
    x = torch.randn(128 * 65535 + 300, 3, generator=gen(2), device=DEV).bfloat16()
    for tile in (1, 128):
        check_quant(x, tile, zpp.quant_fp8(x, tile, transposed=True))


def integers(rows, cols, seed):
    q = torch.randint(-8, 9, (rows, cols), generator=gen(seed), device=DEV).float()
    wide = -(-cols // 16) * 16
    held = torch.empty(rows, wide, dtype=E4M3, device=DEV)
    held.view(torch.uint8).fill_(0x7f)  # NaN behind the rows: not read
    held[:, :cols] = q.to(E4M3)
    return held[:, :cols]


def powers(rows, cols, tile, seed):
    shape = (-(-rows // tile), -(-cols // 128))
    return torch.exp2(torch.randint(-3, 4, shape, generator=gen(seed), device=DEV).float())


def product(a, sa, ta, b, sb, tb):
    va = a.to(torch.float64) * spread(sa, ta, *a.shape)
    vb = b.to(torch.float64) * spread(sb, tb, *b.shape)
    return va @ vb.t(), va.abs() @ vb.abs().t()


SHAPES = [(1, 1, 1), (1, 128, 128), (2, 129, 16), (1, 1000, 2049), (15, 257, 100), (16, 130, 384),
          (17, 128, 129), (33, 300, 1000), (64, 513, 127), (65, 200, 640), (128, 128, 128),
          (129, 127, 1003), (200, 1, 333), (300, 700, 257), (257, 385, 1290), (1000, 129, 48)]


@pytest.mark.parametrize("tiles", [(1, 128), (1, 1), (128, 1), (128, 128)])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product_is_exact_where_fp32_is(m, n, k, tiles):
    ta, tb = tiles
    a, b = integers(m, k, m + k), integers(n, k, n + 2 * k)
    sa, sb = powers(m, k, ta, 3), powers(n, k, tb, 4)
    want, _ = product(a, sa, ta, b, sb, tb)
    for bias in (None, torch.randint(-9, 9, (n,), generator=gen(5), device=DEV).float()):
        y = zpp.matmul_fp8(a, sa, b, sb, bias=bias, dtype=torch.float32)
        assert torch.equal(y.double(), want if bias is None else want + bias.double())
    # scales in another order, rows of y apart: what lies between them stays as it was
    wide = torch.full((m, n + 5), 7.5, device=DEV)
    zpp.matmul_fp8(a, sa.t().contiguous().t(), b, sb.t().contiguous().t(), y=wide[:, 2:n + 2])
    assert torch.equal(wide[:, 2:n + 2].double(), want)
    assert (wide[:, :2] == 7.5).all() and (wide[:, n + 2:] == 7.5).all()
    assert zpp.zpp_device_fault() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n,k,tb", [(1, 4096, 4096, 128), (7, 1000, 3000, 1), (40, 513, 8192, 128),
                                      (300, 520, 4111, 128), (512, 768, 2048, 1), (1024, 4096, 1024, 128)])
def test_product_of_real_data(m, n, k, tb, dtype):
    g = gen(m + n + k)
    x = torch.randn(m, k, generator=g, device=DEV) * torch.exp(torch.randn(k, generator=g, device=DEV))
    w = 0.02 * torch.randn(n, k, generator=g, device=DEV)
    a, sa = zpp.quant_fp8(x.bfloat16())
    b, sb = zpp.quant_fp8(w, tb)
    sa = sa * torch.rand(sa.shape, generator=g, device=DEV)  # any fp32 scales
    bias = torch.randn(n, generator=g, device=DEV).to(dtype)
    want, size = product(a, sa, 1, b, sb, tb)
    want, size = want + bias.double(), size + bias.double().abs()
    y = zpp.matmul_fp8(a, sa, b, sb, bias=bias, dtype=dtype)
    tol = (20 + k / 128) * U * size
    tol = tol + HALF_ULP[dtype] * (want.abs() + tol) + torch.finfo(dtype).smallest_normal * HALF_ULP[dtype]
    assert ((y.double() - want).abs() <= tol).all()
    assert torch.equal(y, zpp.matmul_fp8(a, sa, b, sb, bias=bias, dtype=dtype))  # the same bits


def test_product_with_values_that_are_not_finite():
    a, b = integers(70, 300, 1), integers(140, 300, 2)
    sa, sb = powers(70, 300, 1, 3), powers(140, 300, 128, 4)
    want, _ = product(a, sa, 1, b, sb, 128)
    a[3, 290] = float("nan")
    sa[5, 1] = float("inf")
    sa[6, 2] = 0.0
    y = zpp.matmul_fp8(a, sa, b, sb, dtype=torch.float32).double()
    assert y[3].isnan().all() and not y[5].isfinite().any()
    keep = [i for i in range(70) if i not in (3, 5, 6)]
    assert torch.equal(y[keep], want[keep])
    assert torch.equal(y[6], product(a[6:7], sa[6:7], 1, b, sb, 128)[0][0])


def test_product_forms():
    a, b = integers(24, 300, 1), integers(40, 300, 2)
    sa, sb = powers(24, 300, 1, 3), powers(40, 300, 128, 4)
    want, _ = product(a, sa, 1, b, sb, 128)
    wide = torch.zeros(24, 304, dtype=E4M3, device=DEV)
    wide[:, :300] = a
    y = zpp.matmul_fp8(wide.view(2, 12, 304)[..., :300], sa, b, sb, dtype=torch.float32)
    assert y.shape == (2, 12, 40) and torch.equal(y.view(24, 40).double(), want)
    assert zpp.matmul_fp8(a, sa, b, sb).dtype == torch.bfloat16
    assert zpp.matmul_fp8(a[:0], sa[:0], b, sb).shape == (0, 40)
    assert zpp.matmul_fp8(a, sa, b[:0], sb[:0]).shape == (24, 0)
    same = zpp.matmul_fp8(a, sa, a, sa, dtype=torch.float32)
    assert torch.equal(same.double(), product(a, sa, 1, a, sa, 1)[0])
    # sums at the end of fp16's range: infinite, as a rounding is
    big = torch.full((24, 3), 2.0 ** 20, device=DEV)
    assert zpp.matmul_fp8(a, big, b, sb, dtype=torch.float16).isinf().any()


def test_product_in_a_graph_and_on_streams():
    x = torch.randn(48, 1000, generator=gen(1), device=DEV).bfloat16()
    w = torch.randn(600, 1000, generator=gen(2), device=DEV)
    qw = zpp.quant_fp8(w, 128)
    y = torch.empty(48, 600, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        zpp.matmul_fp8(*zpp.quant_fp8(x), *qw, y=y)
    torch.cuda.current_stream().wait_stream(side)
    want = y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        zpp.matmul_fp8(*zpp.quant_fp8(x), *qw, y=y)
    for k in range(3):
        x.mul_(2.0)
        graph.replay()
        assert torch.equal(y, want * 2.0 ** (k + 1))  # (a power of two moves to the scales)
    # many dependent calls in a row, nothing waited for
    z = x
    for _ in range(20):
        z = zpp.matmul_fp8(*zpp.quant_fp8(z[:, :600] if z.shape[1] != 600 else z),
                           *zpp.quant_fp8(w[:, :600] * 0.04, 128))
    want = x[:, :600]
    for _ in range(20):
        qz, sz = zpp.quant_fp8(want)
        torch.cuda.synchronize()
        qv, sv = zpp.quant_fp8(w[:, :600] * 0.04, 128)
        torch.cuda.synchronize()
        want = zpp.matmul_fp8(qz, sz, qv, sv)
        torch.cuda.synchronize()
    assert torch.equal(z, want)
