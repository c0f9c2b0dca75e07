"""A linear layer whose three products, one forward and two backward, run on e4m3 codes with a scale
per block of 128 (``zpp_quant_fp8``, ``zpp_matmul_fp8``), as a differentiable torch function.
"""
import torch
from torch.autograd.function import once_differentiable

from . import binding as _b


def linear_fp8(x, weight, quantized=None):
    """y = x weight^T, both factors rounded to e4m3 codes: x [..., K] (fp16 / bf16) with a scale for each
    row and 128 columns, weight [N, K] (fp16 / bf16 / fp32) for each 128 x 128 tile. y has x's dtype.

    Differentiable once: with dy rounded like x (along N for dx, along the rows for dweight),
    dx = dy weight in x's dtype and dweight = dy^T x in weight's. A bias is added by the caller.

    quantized: quant_fp8(weight, 128, transposed=True), for a weight that several passes use (micro-
    batches, or answers: there without the transpose). It has to be that of the weight as it is."""
    if not isinstance(x, torch.Tensor) or not isinstance(weight, torch.Tensor):
        raise ValueError("linear_fp8: x and weight are tensors")
    if x.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError(f"x: dtype {x.dtype}, expected float16 or bfloat16")
    if weight.dim() != 2 or x.dim() < 1 or x.shape[-1] != weight.shape[1]:
        raise ValueError(f"weight: {tuple(weight.shape)} does not fit x {tuple(x.shape)}")
    grads = torch.is_grad_enabled() and x.requires_grad
    if quantized is not None:
        if len(quantized) not in (2, 4) or (grads and len(quantized) != 4):
            raise ValueError("quantized: quant_fp8(weight, 128, transposed=True)")
        if tuple(quantized[0].shape) != tuple(weight.shape):
            raise ValueError(f"quantized: codes of {tuple(quantized[0].shape)} do not fit weight")
        if len(quantized) == 4 and tuple(quantized[2].shape) != tuple(weight.shape[::-1]):
            raise ValueError("quantized: quant_fp8(weight, 128, transposed=True)")
    return _Linear.apply(x, weight, quantized)


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, quantized):
        for_x, for_w = ctx.needs_input_grad[:2]
        q = quantized
        if q is None:
            q = _b.quant_fp8(weight, 128, transposed=for_x)
        rows = x.reshape(-1, x.shape[-1])
        qx = _b.quant_fp8(rows, 1, transposed=for_w)
        y = _b.matmul_fp8(qx[0], qx[1], q[0], q[1], dtype=x.dtype)
        ctx.for_x, ctx.for_w = for_x, for_w
        ctx.x_shape, ctx.x_dtype, ctx.w_dtype = x.shape, x.dtype, weight.dtype
        ctx.save_for_backward(*(q[2:] if for_x else (None, None)), *(qx[2:] if for_w else (None, None)))
        return y.view(*x.shape[:-1], weight.shape[0])

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        w_t, w_t_scales, x_t, x_t_scales = ctx.saved_tensors
        rows = dy.reshape(-1, dy.shape[-1]).contiguous()
        qy = _b.quant_fp8(rows, 1, transposed=ctx.for_w)
        dx = dw = None
        if ctx.for_x:
            dx = _b.matmul_fp8(qy[0], qy[1], w_t, w_t_scales, dtype=ctx.x_dtype).view(ctx.x_shape)
        if ctx.for_w and rows.shape[0]:
            dw = _b.matmul_fp8(qy[2], qy[3], x_t, x_t_scales, dtype=ctx.w_dtype)
        elif ctx.for_w:  # no rows: a sum without terms
            dw = dy.new_zeros((dy.shape[-1], ctx.x_shape[-1]), dtype=ctx.w_dtype)
        return dx, dw, None
