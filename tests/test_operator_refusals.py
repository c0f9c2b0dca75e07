"""Argument checks of the AdamW step, the gradient norm and the quantised product: the C
ABI's statuses (fake addresses; every case fails a check before any launch) and the tensor
wrappers' messages. Runs without a GPU."""
import math

import pytest
import torch

import quantized_zero_communication_gb300 as zpp
from quantized_zero_communication_gb300 import binding as zb

OK, INV, MIS, UNS = zb.ZPP_OK, zb.ZPP_ERR_INVALID_ARG, zb.ZPP_ERR_MISALIGNED, zb.ZPP_ERR_UNSUPPORTED
FAKE = 0x10000
cpu_only = pytest.mark.skipif(torch.cuda.is_available(),
                              reason="fake-address cases run only where no GPU exists")


def adamw(n=100, bits=32, g_dt=zb.ZPP_BF16, w_dt=zb.ZPP_BF16, num=None, hp=None, scale=0, **f):
    d = dict(param=FAKE, grad=FAKE, exp_avg=FAKE, exp_avg_sq=FAKE, exp_avg_scale=FAKE,
             exp_avg_sq_scale=FAKE, weight=FAKE)
    d.update(f)
    h = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1, seed=0)
    h.update(hp or {})
    return zb.zpp_adamw_step([zb.AdamwTensor(n=n, **d)] * (1 if num is None else num), g_dt, w_dt,
                             bits, zb.AdamwParams(**h), scale)


@cpu_only
def test_adamw_statuses():
    assert adamw(num=0) == OK and adamw(n=0, param=0, grad=0) == OK
    assert adamw(num=1025, n=0) == INV
    assert adamw(n=-1) == INV and adamw(n=(1 << 38) + 1) == INV
    assert adamw(n=1 << 37, num=3) == INV  # the sum
    for k in ("param", "grad", "exp_avg", "exp_avg_sq"):
        assert adamw(**{k: 0}) == INV
        assert adamw(**{k: FAKE + 8}) == MIS
    assert adamw(weight=FAKE + 8) == MIS
    for k in ("exp_avg_scale", "exp_avg_sq_scale"):
        assert adamw(bits=8, **{k: 0}) == INV
        assert adamw(bits=8, **{k: FAKE + 2}) == MIS
    assert adamw(scale=FAKE + 2) == MIS
    assert adamw(bits=16) == INV and adamw(g_dt=3) == INV and adamw(w_dt=-1) == INV
    assert adamw(w_dt=zb.ZPP_F32) == UNS
    for bad in (dict(lr=math.nan), dict(lr=math.inf), dict(beta1=1.0), dict(beta1=-0.1),
                dict(beta2=1.0), dict(beta2=math.nan), dict(eps=-1e-8), dict(eps=math.inf),
                dict(weight_decay=math.nan), dict(step=0)):
        assert adamw(hp=bad) == INV, bad
    L = zb.lib()
    assert L.zpp_adamw_step(None, 1, 1, 1, 32, zb.ctypes.addressof(zb.AdamwParams()), None, None) == INV
    assert L.zpp_adamw_step(None, 0, 1, 1, 32, None, None, None) == INV


@cpu_only
def test_grad_norm_statuses():
    def call(ptrs=(FAKE,), sizes=(100,), dt=zb.ZPP_F32, pre=1.0, top=1.0, work=FAKE, out=FAKE):
        return zb.zpp_grad_norm(ptrs, sizes, dt, pre, top, work, out)
    assert call(ptrs=[FAKE] * 1025, sizes=[0] * 1025) == INV
    assert call(sizes=(-1,)) == INV and call(sizes=((1 << 38) + 1,)) == INV
    assert call(ptrs=(FAKE, FAKE), sizes=(1 << 37, (1 << 37) + 1)) == INV
    assert call(ptrs=(0,)) == INV and call(work=0) == INV and call(out=0) == INV
    assert call(dt=5) == INV and call(pre=math.inf) == INV
    assert call(top=0.0) == INV and call(top=-1.0) == INV and call(top=math.nan) == INV
    assert call(ptrs=(FAKE + 8,)) == MIS and call(work=FAKE + 2) == MIS and call(out=FAKE + 1) == MIS
    assert zb.lib().zpp_grad_norm(None, None, 1, 2, 1.0, 1.0, FAKE, FAKE, None) == INV
    assert zb.zpp_grad_norm_workspace(-1, 0) == -1 and zb.zpp_grad_norm_workspace(0, -1) == -1
    # room for every tensor's rounded-up chunks
    assert zb.zpp_grad_norm_workspace(16384 * 5, 3) >= 5 + 2


@cpu_only
def test_matvec_statuses():
    def call(rows=8, cols=128, block=64, bits=4, vecs=1, xs=None, ys=None, xd=zb.ZPP_F16,
             yd=zb.ZPP_F32, codes=FAKE, scales=FAKE, x=FAKE, bias=0, y=FAKE):
        return zb.zpp_matvec_blockwise(codes, scales, rows, cols, block, bits, x, xd, vecs,
                                       cols if xs is None else xs, bias, y, yd,
                                       rows if ys is None else ys)
    assert call(rows=0, codes=0, scales=0) == OK and call(vecs=0, x=0, y=0) == OK
    assert call(bits=5) == INV and call(block=32) == INV and call(block=96) == INV
    assert call(cols=0) == INV and call(cols=1 << 31) == INV and call(rows=-1) == INV
    assert call(rows=1 << 31) == INV and call(rows=1 << 30, cols=1 << 9) == INV
    assert call(vecs=-1) == INV and call(vecs=65536) == INV
    assert call(xs=127) == INV and call(ys=7) == INV and call(xs=1 << 39) == INV
    assert call(xd=7) == INV and call(yd=-1) == INV and call(xd=zb.ZPP_F32) == UNS
    for k in ("codes", "scales", "x", "y"):
        assert call(**{k: 0}) == INV
    assert call(codes=FAKE + 8) == MIS and call(x=FAKE + 8) == MIS and call(y=FAKE + 4) == MIS
    assert call(scales=FAKE + 2) == MIS and call(bias=FAKE + 1) == MIS


def z(n, dtype=torch.float32):
    return torch.zeros(n, dtype=dtype)


def raises(match, fn):
    with pytest.raises(ValueError, match=match):
        fn()


F8, BF16, U8 = torch.float8_e4m3fn, torch.bfloat16, torch.uint8


def test_adamw_wrapper_checks():
    def call(p=None, g=None, m=None, v=None, **kw):
        kw = dict(dict(step=1, lr=1e-3), **kw)
        zpp.adamw_step(p if p is not None else z(300), g if g is not None else z(300, BF16),
                       m if m is not None else z(300), v if v is not None else z(300), **kw)
    raises("params: every tensor needs one dtype", lambda: call(p=z(300, BF16)))
    raises("CUDA tensors only", lambda: call())
    raises("at least one tensor", lambda: call(p=[]))
    raises("seed", lambda: call(seed=-1))
    raises("seed", lambda: call(seed=1 << 32))
    raises("at least one tensor", lambda: zpp.grad_norm([]))
    raises("grads: every tensor needs one dtype", lambda: zpp.grad_norm([z(4), z(4, BF16)]))
    raises("grads: every tensor needs one dtype", lambda: zpp.grad_norm([z(4, torch.int32)]))
    raises("CUDA tensors only", lambda: zpp.grad_norm([z(4)]))


def test_optimiser_checks():
    raises("at least one tensor", lambda: zpp.AdamW([]))
    raises("state_bits", lambda: zpp.AdamW([z(4)], state_bits=16))
    raises("come together", lambda: zpp.AdamW([z(4)], exp_avg=[z(4)]))
    raises("scales come with", lambda: zpp.AdamW([z(4)], exp_avg=[z(4)], exp_avg_sq=[z(4)],
                                                 scales=([z(1)], [z(1)])))
    raises("scales come with", lambda: zpp.AdamW([z(4)], state_bits=8, exp_avg=[z(4, F8)],
                                                 exp_avg_sq=[z(4, F8)]))
    raises("seed", lambda: zpp.AdamW([z(4)], seed=1 << 32))
    raises("CUDA tensors only", lambda: zpp.AdamW([z(4)]))


def test_matvec_wrapper_checks():
    x = z(256, torch.float16)
    mv = lambda **k: zpp.matvec_blockwise(**dict(dict(  # noqa: E731
        codes=z(1024, U8), scales=z(32), x=x, rows=8, block=64, bits=4), **k))
    raises("x: dtype", lambda: mv(x=z(256)))
    raises("cols >= 1", lambda: mv(x=z((2, 0), torch.float16)))
    raises("cols >= 1", lambda: mv(rows=-1))
    raises("codes: 1023 elements, expected 1024", lambda: mv(codes=z(1023, U8)))
    raises("codes: dtype", lambda: mv(codes=z(1024)))
    raises("scales: 31 elements, expected 32", lambda: mv(scales=z(31)))
    raises("scales: dtype", lambda: mv(scales=z(32, BF16)))
    raises("bias: dtype", lambda: mv(bias=z(8)))
    raises("bias: 7 elements, expected 8", lambda: mv(bias=z(7, torch.float16)))
    raises("y: 7 elements, expected 8", lambda: mv(y=z(7)))
    raises("y: dtype", lambda: mv(y=z(8, torch.int32)))
    raises("does not fit", lambda: mv(y=z((8, 1))))
    raises("does not fit", lambda: mv(y=z(8), dtype=BF16))
    raises("x: rows must be contiguous", lambda: mv(x=z((512, 2), torch.float16).t()[:, :256]))
    raises("CUDA", lambda: mv())


@pytest.mark.gpu
def test_wrapper_checks_on_the_device():
    """Counts, dtypes and layouts that only matter once the tensors are on the GPU."""
    d = lambda n, dtype=torch.float32: torch.zeros(n, dtype=dtype, device="cuda")  # noqa: E731
    step = lambda **k: zpp.adamw_step(**dict(dict(  # noqa: E731
        params=[d(300)], grads=[d(300)], exp_avg=[d(300)], exp_avg_sq=[d(300)], step=1, lr=1e-3), **k))
    raises("grads: 2 tensors, expected 1", lambda: step(grads=[d(300), d(300)]))
    raises("grads\\[0\\]: 299 elements, expected 300", lambda: step(grads=[d(299)]))
    raises("exp_avg_sq: every tensor needs one dtype", lambda: step(exp_avg_sq=[d(300, BF16)]))
    raises("weights: every tensor needs one dtype", lambda: step(weights=[d(300)]))
    raises("contiguous", lambda: step(grads=[d((300, 2))[:, 0]]))
    raises("CUDA|one device", lambda: step(grads=[z(300)]))
    eight = dict(exp_avg=[d(300, F8)], exp_avg_sq=[d(300, F8)])
    raises("scales\\[0\\]\\[0\\]: 3 elements, expected 2",
           lambda: step(scales=([d(3)], [d(2)]), **eight))
    raises("exp_avg: every tensor needs one dtype", lambda: step(scales=([d(2)], [d(2)])))
    raises("grad_scale: dtype", lambda: step(grad_scale=d(1, BF16)))
    raises("grad_scale: at least", lambda: step(grad_scale=d(0)))
    with pytest.raises(zb.ZppError):
        step(step=0)
    with pytest.raises(zb.ZppError):  # 16-byte alignment
        step(params=[d(301)[1:]])
    opt = zpp.AdamW([d(300)])
    raises("grads\\[0\\]: 10 elements, expected 300", lambda: opt.step([d(10)]))
    raises("replaces", lambda: opt.step([d(300)], max_norm=1.0, grad_scale=d(1)))
    assert opt.steps == 0
    with pytest.raises(zb.ZppError):
        opt.step([d(300)], max_norm=0.0)
    raises("one CUDA device", lambda: zpp.matvec_blockwise(
        d(1024, U8), d(32), z(256, torch.float16), 8, 64, 4))
    with pytest.raises(zb.ZppError):
        zpp.matvec_blockwise(d(1024, U8), d(32), d(264, torch.float16)[4:260], 8, 64, 4)
