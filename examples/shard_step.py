"""One weight through a data-parallel training step and into use, on one GPU.

Four virtual ranks (2 nodes x 2 GPUs) fit W to a teacher's matrix. Every step: each rank's
gradient (its own batch) is reordered and quantised to INT4, reduced over the two hops and averaged
into owner slices; the slices' global norm is clipped and AdamW steps the fp32 master shards
(states in 8 bits), leaving the bf16 weights that the next forward pass uses. At the end the
weights are quantised to INT4 and answer a few single vectors straight from the codes.

    python examples/shard_step.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_zero_communication_gb300 as zpp  # noqa: E402


def main(rows=512, cols=1024, steps=60, batch=256, state_bits=8, device="cuda"):
    """Returns (first loss, last loss, relative error of the INT4 answers)."""
    gen = torch.Generator(device=device).manual_seed(0)
    randn = lambda *s: torch.randn(*s, generator=gen, device=device)  # noqa: E731
    N, M, block = 2, 2, 256
    W, E = N * M, rows * cols  # ranks, weights
    teacher = randn(rows, cols) * 0.02

    # Each rank owns the fp32 masters and states of one slice; the bf16 slices lie back to back,
    # so that the flat buffer is what the all-gather would give every rank.
    flat = torch.zeros(E, dtype=torch.bfloat16, device=device)
    shards = [torch.zeros(E // W, device=device) for _ in range(W)]
    opt = zpp.AdamW(shards, lr=2e-3, weight_decay=0.0, state_bits=state_bits,
                    weights=list(flat.view(W, -1)), seed=1)
    bufs = zpp.QgzBuffers.allocate(W, E, block, 4, M, device)
    grads = torch.empty(W, E, dtype=torch.bfloat16, device=device)
    losses = []
    for _ in range(steps):
        weight, loss = flat.view(rows, cols).float(), 0.0
        for r in range(W):  # forward and backward of every rank's batch
            x = randn(batch, cols)
            err = x @ (weight - teacher).t()
            loss += float(err.square().mean()) / W
            grads[r] = (err.t() @ x / batch).reshape(-1)
        losses.append(loss)
        zpp.qgz_reorder_quant(grads, block, 4, N, M, codes=bufs.c0, scales=bufs.s0)
        zpp.dequant_reduce_requant(bufs.c0, bufs.s0, E, block, 4, N, M, out_codes=bufs.c1,
                                   out_scales=bufs.s1)
        zpp.dequant_reduce_scaled(bufs.c1, bufs.s1, E, block, 4, N, M, out=bufs.out)
        opt.step(list(bufs.out), max_norm=10.0)

    codes, scales = zpp.quant_blockwise(flat, block, 4)
    x = randn(4, cols).bfloat16()
    y = zpp.matvec_blockwise(codes, scales, x, rows, block, 4, dtype=torch.float32)
    want = x.float() @ flat.view(rows, cols).float().t()
    off = float((y - want).norm() / want.norm())
    return losses[0], losses[-1], off


if __name__ == "__main__":
    first, last, off = main()
    print(f"loss {first:.4f} -> {last:.4f} in 60 steps; INT4 answers off by {off:.3f} relative")
