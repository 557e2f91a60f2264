"""One fine-tuning step of several adapters over a shared sparse projection, and a decode step.

    layer norm (keeps its output as an 8-bit checkpoint) -> projection + the tokens' own adapters
    -> backward from the checkpoint -> layer norm backward -> SGD on the adapters

The bf16 activation that the projection reads is dropped after the forward; its backward reads the
checkpoint (33/32 of a byte per element).  Run on an MI355X:

    python examples/multi_adapter_step.py [--tokens 2048] [--hidden 1024] [--ffn 4096] [--rank 16] [--adapters 8]
"""
from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_rank_adapter_amd as sra  # noqa: E402


@dataclass
class Layer:
    """Layer norm, the compressed projection (both directions) and the adapters [n, r, K], [n, N, r]."""
    gamma: torch.Tensor
    beta: torch.Tensor
    Ws: sra.SparseMatrix
    P: sra.SparseMatrix
    A: torch.Tensor
    B: torch.Tensor


def make_layer(K: int, N: int, r: int, n: int, device="cuda", seed: int = 0) -> Layer:
    g = torch.Generator(device=device).manual_seed(seed)
    rand = lambda *s, sd: (torch.randn(*s, generator=g, device=device) * sd).bfloat16()
    Ws, P = sra.compress_pair(rand(N, K, sd=0.02))
    return Layer((1 + rand(K, sd=0.1).float()).bfloat16(), rand(K, sd=0.1), Ws, P, rand(n, r, K, sd=0.02),
                 rand(n, N, r, sd=0.02))


def forward(layer: Layer, H: torch.Tensor, ids: torch.Tensor):
    """Y [T, N] of hidden states H [T, K], and what the backward keeps."""
    X, mean, rstd, kept = sra.layer_norm_fwd(H, layer.gamma, layer.beta, ckpt=True)
    Y, U = sra.multi_lora_fwd(layer.Ws, X, layer.A, layer.B, ids)
    return Y, (H, mean, rstd, kept, U, ids)  # X itself is not kept


def backward(layer: Layer, dY: torch.Tensor, saved, weight_grad: bool = False) -> dict:
    """Gradients of everything the step could train: dH, the adapters, the norm, and (on request) the
    projection's stored values."""
    H, mean, rstd, kept, U, ids = saved
    g = sra.multi_lora_bwd(layer.P, dY, kept, U, layer.A, layer.B, ids)
    if weight_grad:
        g["dW"] = sra.masked_weight_grad(layer.Ws, dY, kept)
    g["dH"], g["dgamma"], g["dbeta"] = sra.layer_norm_bwd(g.pop("dX"), H, layer.gamma, mean, rstd)
    return g


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--ffn", type=int, default=4096)
    ap.add_argument("--rank", type=int, default=16)
    ap.add_argument("--adapters", type=int, default=8)
    ap.add_argument("--steps", type=int, default=10)
    a = ap.parse_args()
    layer = make_layer(a.hidden, a.ffn, a.rank, a.adapters)
    g = torch.Generator(device="cuda").manual_seed(1)
    H = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").bfloat16()
    target = torch.randn(a.tokens, a.ffn, generator=g, device="cuda").bfloat16()
    ids = (torch.arange(a.tokens, device="cuda") * a.adapters // a.tokens).int()  # requests one after another
    lr = 0.1
    for step in range(a.steps):
        Y, saved = forward(layer, H, ids)
        err = Y.float() - target.float()
        grads = backward(layer, (err / a.tokens).bfloat16(), saved)
        layer.A -= (lr * grads["dA"]).bfloat16()
        layer.B -= (lr * grads["dB"]).bfloat16()
        if step % max(1, a.steps // 5) == 0 or step == a.steps - 1:
            print(f"step {step}: loss {0.5 * float((err ** 2).sum(1).mean()):.4f}", flush=True)
    kept = saved[3]
    print(f"kept for the backward: {kept.codes.numel() + kept.exps.numel()} bytes instead of {2 * H.numel()}")
    few = torch.randint(0, a.adapters, (8,), generator=g, device="cuda").int()  # a decode step of 8 requests
    Y, _ = forward(layer, H[:8].contiguous(), few)
    print(f"decode step: {tuple(Y.shape)}")


if __name__ == "__main__":
    main()
