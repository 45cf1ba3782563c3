"""One training step of a pipeline's last stage, from the reconstructed boundary
activation to the loss and back: one attention block and the projection to the
vocabulary, over packed sequences of different lengths.

    h      = w_1 rmsnorm(Xhat), 8 bits                     stage_norm_pack
    q, k, v = h W_qkv^T                                    fp8_gemm
    o      = attention(q, k, v)                            stage_attn
    y      = o W_o^T                                       fp8_pack / fp8_gemm
    X      = s Xhat + gate * w_p rmsnorm(y)
    f      = w_2 rmsnorm(X), 8 bits                        stage_norm_pack
    z      = f W_v^T                                       fp8_gemm
    loss   = cross-entropy and a teacher's top logits      stage_distill

and back to gXhat, which the boundary sends on (mapl_reconstruct_bwd).  The
attention's inputs are columns of one fused projection, and its gradients of that
projection's gradient.  Weights are packed once and would serve all
micro-batches of an optimizer step.

    python examples/last_stage.py [--lengths 700,300,24] [--width d] [--vocab V]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import learned_activation_compression_amd as lac  # noqa: E402


def make(lengths, width: int, heads: int, kv_heads: int, vocab: int, entries: int, seed: int = 0,
         device: str = "cuda") -> dict:
    """Inputs and weights of the step; activations and weights in bf16."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    N, D = sum(lengths), width // heads
    p = dict(Xhat=r(N, width), w_1=1 + 0.1 * r(width), w_p=1 + 0.1 * r(width), gate=0.5 + 0.1 * r(1, width),
             w_2=1 + 0.1 * r(width), W_qkv=r((heads + 2 * kv_heads) * D, width) / width ** 0.5,
             W_o=r(width, width) / width ** 0.5, W_v=r(vocab, width) / width ** 0.5)
    p = {k: v.contiguous().to(device, torch.bfloat16) for k, v in p.items()}
    p["cu"] = torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32).to(device)
    p["labels"] = torch.randint(0, vocab, (N,), generator=g, dtype=torch.int32).to(device)
    p["t_ids"] = torch.randint(0, vocab, (N, entries), generator=g, dtype=torch.int32).to(device)
    p["t_logits"] = (2 * r(N, entries)).to(device)
    p["gloss"] = torch.full((N,), 1.0 / N).to(device)
    return p


def step(p: dict, heads: int, kv_heads: int, temperature: float = 2.0) -> dict:
    """Forward and backward; returns activations and gradients."""
    N, d = p["Xhat"].shape
    D, V = d // heads, p["W_v"].shape[0]
    wide = (heads + 2 * kv_heads) * D
    edge = dict(res_scale=0.8)
    loss_args = dict(labels=p["labels"], t_ids=p["t_ids"], t_logits=p["t_logits"], temperature=temperature, w_ce=0.5,
                     w_kd=0.5 * temperature ** 2)

    def split(x):
        parts = x.split([heads * D, kv_heads * D, kv_heads * D], dim=1)
        return [t.unflatten(1, (-1, D)) for t in parts]

    w8 = {k: lac.fp8_pack(p[k], rows=True, cols=True, square=True) for k in ("W_qkv", "W_o", "W_v")}

    _, h, h8 = lac.stage_norm_pack(p["Xhat"], w_pre=p["w_1"], store_x=False, store_h=True)
    qkv = lac.fp8_gemm(h8, w8["W_qkv"][0], N, wide, d)
    q, k, v = split(qkv)
    o, lse = lac.stage_attn(q, k, v, p["cu"])
    o8, oT8 = lac.fp8_pack(o.flatten(1), rows=True, cols=True)
    y = lac.fp8_gemm(o8, w8["W_o"][0], N, d, d)
    X, f, f8 = lac.stage_norm_pack(p["Xhat"], y, p["w_p"], p["gate"], p["w_2"], **edge, store_h=True)
    z = lac.fp8_gemm(f8, w8["W_v"][0], N, V, d)
    loss, stats = lac.stage_distill(z, **loss_args)

    gz = lac.stage_distill_bwd(p["gloss"], z, stats, **loss_args)
    gz8, gzT8 = lac.fp8_pack(gz, rows=True, cols=True)
    gf = lac.fp8_gemm(gz8, w8["W_v"][1], N, d, V)
    gW_v = lac.fp8_gemm(gzT8, lac.fp8_pack(f, rows=False, cols=True)[1], V, d, N, dtype=torch.float32)
    gx, gy, g_w_p, g_gate, g_w_2 = lac.stage_norm_bwd(gH=gf, X_out=X, Y=y, w_post=p["w_p"], gate=p["gate"],
                                                      w_pre=p["w_2"], **edge)
    gy8, gyT8 = lac.fp8_pack(gy, rows=True, cols=True)
    go = lac.fp8_gemm(gy8, w8["W_o"][1], N, d, d)
    gW_o = lac.fp8_gemm(gyT8, oT8, d, d, N, dtype=torch.float32)
    gqkv = torch.empty_like(qkv)
    gq, gk, gv = split(gqkv)
    lac.stage_attn_bwd(go.unflatten(1, (heads, D)), q, k, v, o, lse, p["cu"], gQ=gq, gK=gk, gV=gv)
    gqkv8, gqkvT8 = lac.fp8_pack(gqkv, rows=True, cols=True)
    gh = lac.fp8_gemm(gqkv8, w8["W_qkv"][1], N, d, wide)
    gW_qkv = lac.fp8_gemm(gqkvT8, lac.fp8_pack(h, rows=False, cols=True)[1], wide, d, N, dtype=torch.float32)
    # the residual's gradient joins that of the norm in front of the block
    gXhat, _, _, _, g_w_1 = lac.stage_norm_bwd(gx, gh, p["Xhat"], w_pre=p["w_1"])
    return dict(h=h, qkv=qkv, o=o.flatten(1), lse=lse, y=y, X=X, f=f, z=z, loss=loss, gz=gz, gf=gf, gx=gx, gy=gy, go=go,
                gqkv=gqkv, gh=gh, gXhat=gXhat, gW_v=gW_v, gW_o=gW_o, gW_qkv=gW_qkv, g_w_p=g_w_p, g_gate=g_gate,
                g_w_2=g_w_2, g_w_1=g_w_1)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--lengths", default="2048,2048,1500,500")
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--vocab", type=int, default=32000)
    a = ap.parse_args()
    heads, kv_heads = a.width // 64, max(1, a.width // 256)
    p = make([int(n) for n in a.lengths.split(",")], a.width, heads, kv_heads, a.vocab, 64)
    step(p, heads, kv_heads)
    e0, e1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    e0.record()
    out = step(p, heads, kv_heads)
    e1.record()
    torch.cuda.synchronize()
    for k, v in out.items():
        print(f"{k:9s} {tuple(v.shape)!s:16s} {str(v.dtype)[6:]:9s} rms {v.double().pow(2).mean().sqrt().item():.4e}")
    print(f"one step: {e0.elapsed_time(e1) * 1e3:.0f} us")


if __name__ == "__main__":
    main()
