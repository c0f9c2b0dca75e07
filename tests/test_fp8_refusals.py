"""Argument checks of the e4m3 quantiser and products: the C ABI's statuses (fake addresses; every case
fails a check before any launch) and the tensor wrappers' messages. Runs without a GPU."""
import ctypes

import pytest
import torch

import quantized_zero_communication_gb300 as zpp
from quantized_zero_communication_gb300 import binding as zb

OK, INV, MIS = zb.ZPP_OK, zb.ZPP_ERR_INVALID_ARG, zb.ZPP_ERR_MISALIGNED
FAKE = 0x10000
E4M3, BF16, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32
cpu_only = pytest.mark.skipif(torch.cuda.is_available(),
                              reason="fake-address cases run only where no GPU exists")


def matrix(**kw):
    d = dict(codes=FAKE, scales=FAKE, rows=64, cols=256, stride=256, scale_row=2, scale_block=1, tile=1)
    d.update(kw)
    return zb.Fp8Matrix(*(d[k] for k, _ in zb.Fp8Matrix._fields_))


BAD = [dict(tile=64), dict(tile=0), dict(rows=-1), dict(rows=1 << 31), dict(cols=0), dict(cols=1 << 31),
       dict(rows=1 << 30, cols=1 << 10, stride=1 << 10), dict(stride=255), dict(stride=(1 << 38) + 16),
       dict(scale_row=-1), dict(scale_block=-1), dict(scale_row=(1 << 38) + 1), dict(codes=0),
       dict(scales=0)]
ASKEW = [dict(codes=FAKE + 8), dict(stride=264), dict(scales=FAKE + 2)]


@cpu_only
def test_quantiser_statuses():
    def call(x=FAKE, dt=zb.ZPP_BF16, x_stride=None, t=None, **kw):
        m = matrix(**kw)
        return zb.zpp_quant_fp8(x, dt, m.cols if x_stride is None else x_stride, m, t)
    assert call(rows=0, x=0, codes=0, scales=0) == OK
    for bad in BAD:
        assert call(**bad) == INV, bad
    for bad in ASKEW:
        assert call(**bad) == MIS, bad
    assert call(x=0) == INV and call(dt=3) == INV and call(x_stride=255) == INV
    assert call(x_stride=(1 << 38) + 1) == INV and call(x=FAKE + 1) == MIS
    assert call(x=FAKE + 2, dt=zb.ZPP_F32) == MIS
    turned = dict(rows=256, cols=64, stride=64)
    for bad in [dict(rows=255), dict(cols=63), dict(tile=128), dict(codes=0), dict(scales=0),
                dict(stride=63)]:
        assert call(t=matrix(**dict(turned, **bad))) == INV, bad
    assert call(t=matrix(**dict(turned, stride=72))) == MIS
    assert call(t=matrix(**dict(turned, codes=FAKE + 4))) == MIS
    L = zb.lib()
    assert L.zpp_quant_fp8(FAKE, 1, 256, None, None, None) == INV


@cpu_only
def test_product_statuses():
    def call(a=None, b=None, bias=0, y=FAKE, dt=zb.ZPP_F32, ys=None):
        b = matrix(**(b or {}))
        return zb.zpp_matmul_fp8(matrix(**(a or {})), b, bias, y, dt, b.rows if ys is None else ys)
    assert call(a=dict(rows=0), y=0) == OK and call(b=dict(rows=0), y=0, ys=0) == OK
    for bad in BAD:
        # (a number of columns that the other matrix does not have is invalid as well)
        assert call(a=bad) == INV, bad
        assert call(b=bad) == INV, bad
    for bad in ASKEW:
        assert call(a=bad) == MIS and call(b=bad) == MIS, bad
    assert call(a=dict(cols=255)) == INV and call(ys=63) == INV and call(ys=(1 << 38) + 1) == INV
    assert call(y=0) == INV and call(dt=3) == INV
    assert call(y=FAKE + 2) == MIS and call(bias=FAKE + 2) == MIS
    assert call(y=FAKE + 1, dt=zb.ZPP_BF16) == MIS and call(bias=FAKE + 1, dt=zb.ZPP_BF16) == MIS
    big = dict(rows=1 << 20, cols=16, stride=16)
    assert call(a=big, b=big) == INV  # more results than ZPP_MAX_ELEMS
    L = zb.lib()
    m = ctypes.addressof(matrix())
    assert L.zpp_matmul_fp8(None, m, None, FAKE, 2, 64, None) == INV
    assert L.zpp_matmul_fp8(m, None, None, FAKE, 2, 64, None) == INV


def raises(match, fn):
    with pytest.raises(ValueError, match=match):
        fn()


def z(shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype)


def test_quantiser_wrapper_checks():
    raises("x: dtype", lambda: zpp.quant_fp8(z((4, 4), torch.int32)))
    raises("tile: 1 or 128", lambda: zpp.quant_fp8(z((4, 4)), 64))
    raises("cols >= 1", lambda: zpp.quant_fp8(z((4, 0))))
    raises("cols >= 1", lambda: zpp.quant_fp8(z(())))
    raises("rows must be contiguous", lambda: zpp.quant_fp8(z((4, 8)).t()))
    raises("evenly spaced", lambda: zpp.quant_fp8(z((4, 5, 8)).transpose(0, 1)))
    raises("a row apart", lambda: zpp.quant_fp8(z(8).as_strided((4, 4), (1, 1))))
    raises("CUDA tensors only", lambda: zpp.quant_fp8(z((4, 4))))


def test_product_wrapper_checks():
    a, sa, b, sb = z((4, 256), E4M3), z((4, 2)), z((200, 256), E4M3), z((2, 2))
    mm = lambda **k: zpp.matmul_fp8(**dict(dict(  # noqa: E731
        a=a, a_scales=sa, b=b, b_scales=sb), **k))
    raises("a: dtype", lambda: mm(a=z((4, 256), torch.uint8)))
    raises("b: dtype", lambda: mm(b=z((200, 256))))
    raises("a_scales: dtype", lambda: mm(a_scales=z((4, 2), BF16)))
    raises("a_scales: .* expected one of", lambda: mm(a_scales=z((4, 3))))
    raises("b_scales: .* expected one of", lambda: mm(b_scales=z((3, 2))))
    raises("b_scales: .* expected one of", lambda: mm(b_scales=z(4)))
    raises("expected .N, 256", lambda: mm(b=z((200, 240), E4M3)))
    raises("expected .N, 256", lambda: mm(b=z((2, 100, 256), E4M3)))
    raises("multiples of 16 bytes", lambda: mm(a=z((4, 250), E4M3)))
    raises("multiples of 16 bytes", lambda: mm(b=z((200, 272), E4M3)[:, 1:257]))
    raises("bias: dtype", lambda: mm(bias=z(200)))
    raises("bias: 199 elements", lambda: mm(bias=z(199, BF16)))
    raises("contiguous", lambda: mm(bias=z(400, BF16)[::2]))
    raises("does not fit", lambda: mm(y=z((4, 199))))
    raises("does not fit", lambda: mm(y=z((4, 200)), dtype=BF16))
    raises("y: dtype", lambda: mm(y=z((4, 200), torch.int32)))
    raises("dtype", lambda: mm(dtype=torch.float64))
    raises("CUDA tensors only", lambda: mm())


def test_linear_wrapper_checks():
    x, w = z((4, 256), BF16), z((200, 256), BF16)
    raises("x: dtype", lambda: zpp.linear_fp8(z((4, 256)), w))
    raises("does not fit x", lambda: zpp.linear_fp8(x, z((200, 255), BF16)))
    raises("does not fit x", lambda: zpp.linear_fp8(x, z(256, BF16)))
    raises("does not fit x", lambda: zpp.linear_fp8(z((4, 0), BF16), z((200, 0), BF16)))
    raises("tensors", lambda: zpp.linear_fp8(x, None))
    raises("quantized", lambda: zpp.linear_fp8(x, w, quantized=(w,)))
    raises("do not fit weight", lambda: zpp.linear_fp8(x, w, quantized=(x, x)))
    raises("quantized", lambda: zpp.linear_fp8(z((4, 256), BF16).requires_grad_(), w, quantized=(w, w)))
    raises("CUDA tensors only", lambda: zpp.linear_fp8(x, w))
