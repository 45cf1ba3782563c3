"""Tensors whose offsets pass 2^31 and 2^32: the operators against themselves on
the last rows alone (rows are independent, and a row's mask is a function of its
counter), and against exact integer products."""
import pytest
import torch

import learned_activation_compression_amd as lac

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_dropout_beyond_2_to_32_elements():
    N, d = 65541, 65537  # 4.3e9 elements, odd rows
    X = torch.full((N, d), 1.0, dtype=torch.bfloat16, device=DEV)
    Y = lac.stage_dropout(X, 0.25, 7, 11)
    for r in (0, 32768, N - 3):
        assert torch.equal(Y[r:r + 3], lac.stage_dropout(X[r:r + 3].contiguous(), 0.25, 7, 11 + r))


def test_edge_beyond_2_to_31_elements():
    N, d = 300_003, 8192  # 2.5e9 elements
    g = torch.Generator(device=DEV).manual_seed(1)
    X = torch.randn(N, d, dtype=torch.bfloat16, device=DEV, generator=g)
    w = torch.full((d,), 0.5, dtype=torch.bfloat16, device=DEV)
    kw = dict(res_scale=0.5, p=0.1, seed=3)
    x, h = lac.stage_norm(X, X, w, None, w, **kw, offset=0)
    gX, gY, gp, _, gq = lac.stage_norm_bwd(X, h, x, X, w, None, w, **kw, offset=0)
    for r in (0, 262_144, N - 2):
        s = slice(r, r + 2)
        x2, h2 = lac.stage_norm(X[s], X[s], w, None, w, **kw, offset=r)
        assert torch.equal(x[s], x2) and torch.equal(h[s], h2)
        a, b, *_ = lac.stage_norm_bwd(X[s], h[s], x[s], X[s], w, None, w, **kw, offset=r)
        assert torch.equal(gX[s], a) and torch.equal(gY[s], b)
    assert gp.isfinite().all() and gq.isfinite().all()


def test_products_beyond_2_to_31_elements():
    M, N, K = 66_001, 33_003, 128  # C: 2.2e9 elements
    g = torch.Generator(device=DEV).manual_seed(2)
    A = torch.randint(-2, 3, (M, K), device=DEV, generator=g).bfloat16()
    B = torch.randint(-2, 3, (N, K), device=DEV, generator=g).bfloat16()
    C = lac.fp8_gemm(lac.fp8_pack(A)[0], lac.fp8_pack(B)[0], M, N, K)
    for r in (0, 40_000, M - 256):
        want = A[r:r + 256].float() @ B.float().t().contiguous()
        assert torch.equal(C[r:r + 256].float(), want.bfloat16().float())


def test_packs_beyond_2_to_31_elements():
    R, C = 262_200, 8200  # 2.15e9 elements
    X = torch.zeros(R, C, dtype=torch.bfloat16, device=DEV)
    X[-3:] = torch.arange(C, device=DEV) % 8
    X[:, -1] = 3.0
    pk, pkT = lac.fp8_pack(X, rows=True, cols=True)
    V = lac.fp8_unpack(pk, R, C, torch.bfloat16)
    assert torch.equal(V[-200:], X[-200:]) and torch.equal(V[:200], X[:200])
    del V
    T = lac.fp8_unpack(pkT, C, R, torch.bfloat16)
    assert torch.equal(T[-100:, -300:], X[-300:, -100:].t()) and torch.equal(T[:100, -300:], X[-300:, :100].t())
