"""A linear layer whose three products, one forward and two backward, run on e4m3 codes with a scale
per block of 128 (``zpp_quant_fp8``, ``zpp_matmul_fp8``), as a differentiable torch function (whose
passes are in the extension ``_tensors``).
"""
import torch

from . import binding as _b


def linear_fp8(x, weight, quantized=None):
    """y = x weight^T, both factors rounded to e4m3 codes: x [..., K] (fp16 / bf16) with a scale for each
    row and 128 columns, weight [N, K] (fp16 / bf16 / fp32) for each 128 x 128 tile. y has x's dtype.

    Differentiable once: with dy rounded like x (along N for dx, along the rows for dweight),
    dx = dy weight in x's dtype and dweight = dy^T x in weight's. A bias is added by the caller.
    A captured backward pass raises while a graph made on the default stream holds x or weight.

    quantized: quant_fp8(weight, 128, transposed=True), for a weight that several passes use (micro-
    batches, or answers: there without the transpose). It has to be that of the weight as it is."""
    if not isinstance(x, torch.Tensor) or not isinstance(weight, torch.Tensor):
        raise ValueError("linear_fp8: x and weight are tensors")
    if x.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError(f"x: dtype {x.dtype}, expected float16 or bfloat16")
    if weight.dim() != 2 or x.dim() < 1 or x.shape[-1] != weight.shape[1] or not weight.shape[1]:
        raise ValueError(f"weight: {tuple(weight.shape)} does not fit x {tuple(x.shape)}")
    grads = torch.is_grad_enabled() and x.requires_grad
    if quantized is not None:
        if len(quantized) not in (2, 4) or (grads and len(quantized) != 4):
            raise ValueError("quantized: quant_fp8(weight, 128, transposed=True)")
        if tuple(quantized[0].shape) != tuple(weight.shape):
            raise ValueError(f"quantized: codes of {tuple(quantized[0].shape)} do not fit weight")
        if len(quantized) == 4 and tuple(quantized[2].shape) != tuple(weight.shape[::-1]):
            raise ValueError("quantized: quant_fp8(weight, 128, transposed=True)")
        if weight.shape[0]:  # (the codes of a weight without rows have no columns in their transpose)
            for name, codes, scales, tile in zip(("codes", "codes_t"), quantized[::2], quantized[1::2], (128, 128)):
                _b._fp8(codes, scales, name, tile)
        quantized = tuple(quantized)
    _b._on_gpu(x, weight, *(quantized or ()))
    return _b._tensors().linear_fp8(_b._address("zpp_quant_fp8"), _b._address("zpp_matmul_fp8"), x, weight,
                                    quantized)
