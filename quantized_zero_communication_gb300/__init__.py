"""GB300 (sm_103a) ZeRO++ block-quantisation hot path: qwZ quantise / dequantise and
the qgZ reorder-quantise, fused intra-node dequant-reduce-requant and final
dequant-reduce, and on either side of them the AdamW step with its gradient norm, the Muon step,
the product with quantised weights and the products of a linear layer in fp8, behind the C ABI
declared in ``include/zpp.h``.

``binding`` is the ctypes layer over ``libzpp.so``; ``optim`` the optimisers; ``linear`` the linear layer;
``inputs`` holds the seeded synthetic workloads. The library is loaded on first use.
"""
from .binding import (  # noqa: F401
    Fp8Matrix, LocalRange, QgzBuffers, Topology, ZppError, adamw_step, dequant_blockwise,
    dequant_reduce, dequant_reduce_local, dequant_reduce_requant, dequant_reduce_requant_local,
    dequant_reduce_scaled, device_copy, grad_norm, matmul_fp8, matvec_blockwise, orthogonalize,
    qgz_pipelined, qgz_reorder_quant, qgz_reorder_quant_local, qgz_reorder_quant_tensors,
    quant_blockwise, quant_fp8, zpp_code_bytes, zpp_device_fault, zpp_num_scales, zpp_status_string)
from .optim import AdamW, Muon  # noqa: F401


def __getattr__(name):  # (what needs torch when it is imported)
    if name == "linear_fp8":
        from .linear import linear_fp8
        globals()[name] = linear_fp8
        return linear_fp8
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
