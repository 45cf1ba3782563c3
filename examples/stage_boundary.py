"""One training step of two pipeline stages around a compressed boundary.

Sending stage, end of its last block (x is the residual stream, a the block's
inner activation):

    y     = a W_out^T                      8-bit product, fp8_pack / fp8_gemm
    X     = s x + gate * rmsnorm(dropout(y))          stage_norm
    Z     = (X - E[t] P) A                            mapl_compress

Receiving stage, head of its first block:

    Xhat  = Z A^T + E[t] P                            mapl_reconstruct
    h     = w * rmsnorm(Xhat)                         stage_norm
    q     = dropout(h W_in^T)                         8-bit product, stage_dropout

and back from a loss gradient dL/dq: the receiver's products, norm and
reconstruct gradients, the boundary gradient gZ, then the sender's compress,
block-edge and product gradients.  Masks come from (seed, row): nothing of them
is stored.  Weights are packed once and would serve all micro-batches of an
optimizer step.

    python examples/stage_boundary.py [--tokens N] [--width d] [--rank r]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import learned_activation_compression_amd as lac  # noqa: E402


def orthonormal(rows: int, cols: int, gen) -> torch.Tensor:
    return torch.linalg.qr(torch.randn(max(rows, cols), min(rows, cols), generator=gen))[0]


def make(tokens: int, width: int, rank: int, vocab: int = 1000, seed: int = 0, device: str = "cuda") -> dict:
    """Inputs and weights of the step, bf16."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    p = dict(x=r(tokens, width), a=r(tokens, width), W_out=r(width, width) / width ** 0.5,
             W_in=r(width, width) / width ** 0.5, w_post=1 + 0.1 * r(width), gate=0.5 + 0.1 * r(1, width),
             w_pre=1 + 0.1 * r(width), E=0.1 * r(vocab, rank), P=orthonormal(width, rank, g).t().contiguous(),
             A=orthonormal(width, rank, g), gq=r(tokens, width) / tokens)
    p = {k: v.contiguous().to(device, torch.bfloat16) for k, v in p.items()}
    p["tids"] = torch.randint(0, vocab, (tokens,), generator=g, dtype=torch.int32).to(device)
    return p


def step(p: dict, drop: float = 0.1, seed: int = 1234, first_row: int = 0) -> dict:
    """Forward and backward; returns activations and gradients."""
    N, d = p["x"].shape
    edge = dict(res_scale=0.8, p=drop, seed=seed, offset=first_row)
    tids, E, P, A = p["tids"], p["E"], p["P"], p["A"]
    out8, outT8 = lac.fp8_pack(p["W_out"], rows=True, cols=True, square=True)
    in8, inT8 = lac.fp8_pack(p["W_in"], rows=True, cols=True, square=True)

    # sender, forward
    a8, aT8 = lac.fp8_pack(p["a"], rows=True, cols=True)
    y = lac.fp8_gemm(a8, out8, N, d, d)
    X, _ = lac.stage_norm(p["x"], y, p["w_post"], p["gate"], **edge)
    Z = lac.mapl_compress(X, tids, E, P, A)
    # receiver, forward
    Xhat = lac.mapl_reconstruct(Z, tids, E, P, A)
    _, h = lac.stage_norm(Xhat, w_pre=p["w_pre"], store_x=False)
    h8, hT8 = lac.fp8_pack(h, rows=True, cols=True)
    q = lac.stage_dropout(lac.fp8_gemm(h8, in8, N, d, d), drop, seed + 1, first_row)
    # receiver, backward
    gz = lac.stage_dropout(p["gq"], drop, seed + 1, first_row)
    gz8, gzT8 = lac.fp8_pack(gz, rows=True, cols=True)
    gh = lac.fp8_gemm(gz8, inT8, N, d, d)
    gW_in = lac.fp8_gemm(gzT8, hT8, d, d, N, dtype=torch.float32)
    gXhat, _, _, _, g_w_pre = lac.stage_norm_bwd(gH=gh, X_out=Xhat, w_pre=p["w_pre"])
    gZ, gA = lac.mapl_reconstruct_bwd(gXhat, Z, A)
    # sender, backward
    gX, gA = lac.mapl_compress_bwd(gZ, X, tids, E, P, A, gA=gA, accumulate=True)
    gx, gy, g_w_post, g_gate, _ = lac.stage_norm_bwd(gX, Y=y, w_post=p["w_post"], gate=p["gate"], **edge)
    gy8, gyT8 = lac.fp8_pack(gy, rows=True, cols=True)
    ga = lac.fp8_gemm(gy8, outT8, N, d, d)
    gW_out = lac.fp8_gemm(gyT8, aT8, d, d, N, dtype=torch.float32)
    return dict(y=y, X=X, Z=Z, Xhat=Xhat, h=h, q=q, gz=gz, gh=gh, gXhat=gXhat, gZ=gZ, gX=gX, gx=gx, gy=gy, ga=ga,
                gW_out=gW_out, gW_in=gW_in, gA=gA, g_w_post=g_w_post, g_gate=g_gate, g_w_pre=g_w_pre)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--rank", type=int, default=128)
    a = ap.parse_args()
    p = make(a.tokens, a.width, a.rank)
    step(p)
    e0, e1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    e0.record()
    out = step(p)
    e1.record()
    torch.cuda.synchronize()
    for k, v in out.items():
        print(f"{k:9s} {tuple(v.shape)!s:16s} {str(v.dtype)[6:]:9s} rms {v.double().pow(2).mean().sqrt().item():.4e}")
    print(f"one step: {e0.elapsed_time(e1) * 1e3:.0f} us")


if __name__ == "__main__":
    main()
