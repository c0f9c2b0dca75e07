"""One linear layer in fp8, trained by Muon, on one GPU.

The layer's matrix fits a teacher's. Every step: its three products run on e4m3 codes with a scale per
block of 128 (the weight's codes serve two micro-batches), Muon steps the fp32 master with the clipped
gradient, and the new bf16 weight goes to codes again. At the end one token is answered from the codes.

    python examples/fp8_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_zero_communication_gb300 as zpp  # noqa: E402


def main(rows=512, cols=1024, steps=40, batch=256, device="cuda"):
    """Returns (first loss, last loss, relative error of the token's answer)."""
    gen = torch.Generator(device=device).manual_seed(0)
    randn = lambda *s: torch.randn(*s, generator=gen, device=device)  # noqa: E731
    teacher = randn(rows, cols) * 0.02
    master = torch.zeros(rows, cols, device=device)
    weight = torch.zeros(rows, cols, dtype=torch.bfloat16, device=device, requires_grad=True)
    opt = zpp.Muon([master], lr=5e-3, weight_decay=0.0, adjust="match_rms_adamw",
                   weights=[weight.detach()])
    codes = zpp.quant_fp8(weight.detach(), 128, transposed=True)
    losses = []
    for _ in range(steps):
        loss, grad = 0.0, torch.zeros(rows, cols, device=device)
        for _ in range(2):  # micro-batches
            x = randn(batch, cols).bfloat16()
            y = zpp.linear_fp8(x, weight, quantized=codes)
            error = y.float() - x.float() @ teacher.t()
            part = error.square().mean()
            grad += torch.autograd.grad(part, weight)[0].float()
            loss += float(part.detach()) / 2
        losses.append(loss)
        opt.step([grad], max_norm=1.0, pre_scale=0.5)
        zpp.quant_fp8(weight.detach(), 128, transposed=True, out=codes)
    token = randn(1, cols).bfloat16()
    y = zpp.matmul_fp8(*zpp.quant_fp8(token), codes[0], codes[1], dtype=torch.float32)
    want = token.float() @ weight.detach().float().t()
    return losses[0], losses[-1], float((y - want).detach().norm() / want.norm())


if __name__ == "__main__":
    first, last, off = main()
    print(f"loss {first:.4f} -> {last:.4f} in 40 steps; the token's answer off by {off:.3f} relative")
