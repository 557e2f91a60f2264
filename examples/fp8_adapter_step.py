"""One fine-tuning step of a block with an 8-bit dense projection and a sparse one with an adapter.

    H = X + R, root-mean-square norm (writes Y and its 8-bit form in one pass)
    -> up = Y W^T in 8-bit floating point -> ReLU -> sparse projection + low-rank adapter
    -> backward: the sparse layer's, then two 8-bit products (input and weight gradient), the norm's
    -> update: the adapter's gradients orthogonalised, the dense weight by its gradient and coded again

Run on an MI355X:

    python examples/fp8_adapter_step.py [--tokens 2048] [--hidden 1024] [--ffn 4096] [--rank 16]
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
class Block:
    """The norm's weight, the dense up projection W [F, K] with its 8-bit form and that of its transpose, the sparse
    down projection (both directions) and its adapter A [r, F], B [K, r]."""
    gamma: torch.Tensor
    W: torch.Tensor
    W8: sra.Fp8Matrix
    W8t: sra.Fp8Matrix
    Ws: sra.SparseMatrix
    P: sra.SparseMatrix
    A: torch.Tensor
    B: torch.Tensor


def make_block(K: int, F: int, r: int, device="cuda", seed: int = 0) -> Block:
    g = torch.Generator(device=device).manual_seed(seed)
    rand = lambda *s, sd: (torch.randn(*s, generator=g, device=device) * sd).bfloat16()
    W = rand(F, K, sd=K ** -0.5)
    Ws, P = sra.compress_pair(rand(K, F, sd=F ** -0.5))
    return Block((1 + rand(K, sd=0.1).float()).bfloat16(), W, *sra.fp8_encode_pair(W, block_rows=128), Ws, P,
                 rand(r, F, sd=F ** -0.5), rand(K, r, sd=0.02))


def forward(blk: Block, X: torch.Tensor, R: torch.Tensor):
    """The block's output [T, K], H = X + R, and what the backward keeps."""
    Y, H, rstd, Y8 = sra.rms_norm_fwd(X, blk.gamma, residual=R, fp8=torch.float8_e4m3fn)
    act = sra.fp8_matmul(Y8, blk.W8).clamp_(min=0)
    out, U = sra.sparse_lora_fwd(blk.Ws, act, blk.A, blk.B)
    return out, H, (Y, H, rstd, act, U)


def backward(blk: Block, dOut: torch.Tensor, dH: torch.Tensor | None, saved) -> dict:
    """Gradients: dX (of X and of the residual alike), dgamma, dW (fp32), dA and dB."""
    Y, H, rstd, act, U = saved
    g = sra.sparse_lora_bwd(blk.P, dOut, act, U, blk.A, blk.B)
    g["dUp"] = g.pop("dX") * (act > 0)
    d8, d8t = sra.fp8_encode_pair(g["dUp"], torch.float8_e5m2)
    g["dY"] = sra.fp8_matmul(d8, blk.W8t)
    g["dW"] = sra.fp8_matmul(d8t, sra.fp8_encode_t(Y), out_dtype=torch.float32)
    g["dX"], g["dgamma"] = sra.rms_norm_bwd(g["dY"], H, blk.gamma, rstd, dH=dH)
    return g


def update(blk: Block, g: dict, lr: float):
    """The adapter moves along its orthogonalised gradients, the dense weight along its gradient."""
    blk.A -= (lr * sra.orthogonalize(g["dA"])).bfloat16()
    blk.B -= (lr * sra.orthogonalize(g["dB"])).bfloat16()
    blk.W -= (lr * g["dW"]).bfloat16()
    sra.fp8_encode_pair(blk.W, block_rows=128, out=(blk.W8, blk.W8t))


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--ffn", type=int, default=4096)
    ap.add_argument("--rank", type=int, default=16)
    ap.add_argument("--steps", type=int, default=10)
    a = ap.parse_args()
    blk = make_block(a.hidden, a.ffn, a.rank)
    g = torch.Generator(device="cuda").manual_seed(1)
    X, R, target = (torch.randn(a.tokens, a.hidden, generator=g, device="cuda").bfloat16() for _ in range(3))
    for step in range(a.steps):
        out, _, saved = forward(blk, X, R)
        err = out.float() - target.float()
        update(blk, backward(blk, (err / a.tokens).bfloat16(), None, saved), lr=0.01)
        if step % max(1, a.steps // 5) == 0 or step == a.steps - 1:
            print(f"step {step}: loss {0.5 * float((err ** 2).sum(1).mean()):.4f}", flush=True)
    held = sum(m.codes.numel() + m.exps.numel() for m in (blk.W8, blk.W8t))
    print(f"dense weight, both directions: {held} bytes in 8 bits")
    few = torch.randn(8, a.hidden, generator=g, device="cuda").bfloat16()  # a decode step of 8 requests
    print(f"decode step: {tuple(forward(blk, few, torch.zeros_like(few))[0].shape)}")


if __name__ == "__main__":
    main()
