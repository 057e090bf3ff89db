"""Train a pre-norm MoE block on a fixed target, put its experts into 4 bits, and decode with it.

    python examples/block_train_and_decode.py [--tokens 512] [--hidden 512] [--ffn 256] [--experts 16] [--top-k 2]
                                              [--steps 30] [--state-bits 8] [--group 64]

Runs the whole of the block: add + RMSNorm and its backward, the padding-free layer's step, AdamW with 8-bit (or 32-bit)
states, the quantisation, and a decode step (norm with 8-bit output, router, 4-bit experts) for single tokens.
"""

from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mixture_experts_layer_pft_gb300 import block, build  # noqa: E402


def make_params(h, f, E, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s, std: torch.randn(*s, generator=g, device="cuda") * std  # noqa: E731
    return {"gamma": torch.ones(h, device="cuda"), "Wg": rn(h, E, std=1 / math.sqrt(h)), "bias": None,
            "W1": rn(E, h, f, std=1 / math.sqrt(h)).to(dtype), "W3": rn(E, h, f, std=1 / math.sqrt(h)).to(dtype),
            "W2": rn(E, f, h, std=1 / math.sqrt(f)).to(dtype)}


def train(params, T, k, steps, bits, lr=2e-3, seed=1):
    """Losses of `steps` steps towards a fixed random target of s + y; the buffers hold the last step."""
    E, h, f = params["W1"].shape
    dt = params["W1"].dtype
    b = block.BlockBuffers(T, h, E, k, f, dt)
    opt = block.AdamW(*block.parameters(params, b), lr=lr, bits=bits, weight_decay=[0.0, 0.0, 0.01, 0.01, 0.01])
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, residual, target = (torch.randn(T, h, generator=g, device="cuda").to(dt) for _ in range(3))
    losses = []
    for _ in range(steps):
        y, s = block.block_forward(params, x, residual, b)
        error = s.float() + y.float() - target.float()
        losses.append(error.square().mean())
        d = (2.0 / T * error).to(dt)  # of the summed squares: per-token gradients of order one
        block.block_backward(params, d, d, b)
        opt.step()
    return [float(v) for v in losses], b, (x, residual)


def decode(params, x, residual, k, group, act8=True):
    """y of the tokens one by one, from 4-bit experts."""
    dec = block.DecodeBlock(params, 1, k, group=group, act8=act8)
    return torch.cat([dec.step(x[t:t + 1].contiguous(), residual[t:t + 1].contiguous())[0].clone() for t in range(x.shape[0])])


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 512), ("hidden", 512), ("ffn", 256), ("experts", 16), ("top-k", 2), ("steps", 30),
                        ("state-bits", 8), ("group", 64)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args(argv)
    build.build()
    params = make_params(a.hidden, a.ffn, a.experts, torch.bfloat16)
    losses, b, (x, residual) = train(params, a.tokens, a.top_k, a.steps, a.state_bits)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps with {a.state_bits}-bit states")
    n = min(a.tokens, 8)
    y, _ = block.block_forward(params, x, residual, b)
    y4 = decode(params, x[:n], residual[:n], a.top_k, a.group)
    off = float((y4.float() - y[:n].float()).norm() / y[:n].float().norm())
    print(f"{n} tokens decoded from 4-bit experts: {off:.3f} of the bf16 layer's outputs off")
    return losses, off


if __name__ == "__main__":
    main()
