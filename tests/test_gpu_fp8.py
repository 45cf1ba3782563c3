"""8-bit packs and products on the GPU against the float64 oracle.

Tolerances.  A pack's values are whole numbers of quanta: they equal the
oracle's.  A product of integers with sums below 2^24 is exact whatever the
order.  Otherwise K products add up in fp32, each addition off by one step at
most (the matrix cores may truncate), and the result is rounded once to its
type."""
import numpy as np
import pytest
import torch

import learned_activation_compression_amd as lac
from oracle import stage

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def n64(t):
    return t.detach().cpu().double().numpy()


def data(R, C, dt, seed=0):
    rng = np.random.default_rng(seed + 10007 * R + C)
    x = rng.standard_normal((R, C)) * np.exp(2 * rng.standard_normal((R, 1))) * np.exp(rng.standard_normal(C))
    x.reshape(-1)[rng.integers(0, R * C, max(1, R * C // 50))] = 0
    return torch.from_numpy(x.astype(np.float32)).to(DT[dt]).to(DEV)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("square", [False, True])
@pytest.mark.parametrize("R, C", [(1, 1), (1, 128), (31, 17), (33, 129), (128, 128), (130, 257), (200, 1000), (257, 64)])
def test_pack_values(R, C, square, dt):
    X = data(R, C, dt)
    pk, pkT = lac.fp8_pack(X, rows=True, cols=True, square=square)
    x = n64(X)
    assert np.array_equal(n64(lac.fp8_unpack(pk, R, C)), stage.round_blocks(x, square))
    want_t = stage.round_blocks(np.ascontiguousarray(x.T), square)
    assert np.array_equal(n64(lac.fp8_unpack(pkT, C, R)), want_t)
    assert np.array_equal(n64(lac.fp8_unpack(pkT, C, R, torch.bfloat16)), want_t)  # 4 bits fit bf16
    # each alone
    only, none = lac.fp8_pack(X, rows=True, cols=False, square=square)
    assert none is None and torch.equal(lac.fp8_unpack(only, R, C), lac.fp8_unpack(pk, R, C))
    none, only = lac.fp8_pack(X, rows=False, cols=True, square=square)
    assert none is None and torch.equal(lac.fp8_unpack(only, C, R), lac.fp8_unpack(pkT, C, R))


def test_pack_extremes():
    X = torch.zeros(4, 640, device=DEV)
    X[0, :128] = torch.linspace(-448, 448, 128, device=DEV)
    X[0, 128] = 3.0e38                       # the largest scales
    X[0, 129] = -1.0
    X[1, :3] = torch.tensor([1e-38, 1e-42, -3e-45], device=DEV)
    X[2, 5], X[2, 6], X[2, 7] = float("inf"), float("nan"), 2.0
    X[3, 300] = 1.76 * 2.0 ** 20             # just above 448 * 2^12
    X[3, 301] = 1.75 * 2.0 ** 8
    for sq in (False, True):
        pk, pkT = lac.fp8_pack(X, rows=True, cols=True, square=sq)
        x = n64(X)
        a, b = n64(lac.fp8_unpack(pk, 4, 640)), n64(lac.fp8_unpack(pkT, 640, 4))
        assert np.array_equal(a, stage.round_blocks(x, sq), equal_nan=True)
        assert np.array_equal(b, stage.round_blocks(np.ascontiguousarray(x.T), sq), equal_nan=True)
        assert np.isnan(a[2, 5]) and np.isnan(a[2, 6]) and np.isfinite(np.delete(a.reshape(-1), [1285, 1286])).all()


SHAPES = [(1, 1, 1), (1, 32, 128), (7, 100, 5), (32, 64, 130), (33, 31, 1000), (64, 500, 256), (65, 129, 127),
          (128, 128, 128), (129, 257, 384), (200, 1000, 640), (300, 520, 2048), (1000, 96, 16), (16, 2048, 2048),
          (1000, 1530, 1999), (520, 520, 9000), (16, 16, 16384), (64, 90, 9000), (100, 300, 8200), (128, 140, 8191)]


@pytest.mark.parametrize("M, N, K", SHAPES)
def test_integer_products_are_exact(M, N, K):
    # |a|, |b| <= 2: sums below 4 K < 2^24; a different power of two scales each row's block
    rng = np.random.default_rng(M + N + K)
    a, b = rng.integers(-2, 3, (M, K)), rng.integers(-2, 3, (N, K))
    want = a @ b.T
    A, B = (torch.from_numpy(v.astype(np.float32)).to(DEV) for v in (a, b))
    pa, pb = lac.fp8_pack(A)[0], lac.fp8_pack(B)[0]
    C = lac.fp8_gemm(pa, pb, M, N, K, dtype=torch.float32)
    assert np.array_equal(n64(C), want)
    lac.fp8_gemm(pa, pb, M, N, K, C=C, accumulate=True)
    assert np.array_equal(n64(C), 2 * want)
    bf = lac.fp8_gemm(pa, pb, M, N, K)
    assert torch.equal(bf, torch.from_numpy(want.astype(np.float32)).to(DEV).bfloat16())
    # rows scaled by powers of two, exactly representable all the same
    sa, sb = 2.0 ** rng.integers(-20, 20, (M, 1)), 2.0 ** rng.integers(-20, 20, (N, 1))
    pa, pb = lac.fp8_pack(A * torch.from_numpy(sa).float().to(DEV))[0], lac.fp8_pack(B * torch.from_numpy(sb).float().to(DEV))[0]
    assert np.array_equal(n64(lac.fp8_gemm(pa, pb, M, N, K, dtype=torch.float32)), want * sa * sb.T)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("M, N, K", [(5, 70, 1000), (190, 300, 700), (1000, 512, 1536), (513, 260, 4100)])
def test_products_with_block_scales(M, N, K, dt):
    A, B = data(M, K, dt, 1), data(N, K, dt, 2)
    a = stage.round_blocks(n64(A))
    b = stage.round_blocks(n64(B), square=True)
    C = lac.fp8_gemm(lac.fp8_pack(A)[0], lac.fp8_pack(B, square=True)[0], M, N, K, dtype=DT[dt])
    ref, size = a @ b.T, np.abs(a) @ np.abs(b).T
    bound = torch.finfo(DT[dt]).eps / 2 * np.abs(ref) * (1 + 2.0 ** -7) + K * torch.finfo(torch.float32).eps * size
    err = np.abs(n64(C) - ref)
    assert (err <= bound).all(), float((err / np.maximum(bound, 1e-300)).max())


def test_linear_layer_forward_and_backward():
    # the three products of a projection from packs of X, W, gY and their transposes, each tensor read once
    N, K, M = 300, 200, 330
    X, W, gY = data(N, K, "bf16", 3), data(M, K, "bf16", 4), data(N, M, "bf16", 5)
    x8, xT8 = lac.fp8_pack(X, rows=True, cols=True)
    w8, wT8 = lac.fp8_pack(W, rows=True, cols=True, square=True)
    g8, gT8 = lac.fp8_pack(gY, rows=True, cols=True)
    x, xT = stage.round_blocks(n64(X)), stage.round_blocks(np.ascontiguousarray(n64(X).T))
    w = stage.round_blocks(n64(W), square=True)
    g, gT = stage.round_blocks(n64(gY)), stage.round_blocks(np.ascontiguousarray(n64(gY).T))
    for got, a, b in ((lac.fp8_gemm(x8, w8, N, M, K, dtype=torch.float32), x, w),
                      (lac.fp8_gemm(g8, wT8, N, K, M, dtype=torch.float32), g, w.T),
                      (lac.fp8_gemm(gT8, xT8, M, K, N, dtype=torch.float32), gT, xT)):
        bound = a.shape[1] * torch.finfo(torch.float32).eps * (np.abs(a) @ np.abs(b).T)
        assert (np.abs(n64(got) - a @ b.T) <= bound).all()


def test_values_that_are_not_finite_reach_their_rows_only():
    M, N, K = 70, 90, 300
    A, B = data(M, K, "f32", 6), data(N, K, "f32", 7)
    clean = lac.fp8_gemm(lac.fp8_pack(A)[0], lac.fp8_pack(B)[0], M, N, K, dtype=torch.float32)
    A[40, 7], B[66, 250] = float("inf"), float("nan")
    C = lac.fp8_gemm(lac.fp8_pack(A)[0], lac.fp8_pack(B)[0], M, N, K, dtype=torch.float32)
    assert C[40].isnan().all() and C[:, 66].isnan().all()
    rm, rn = [i for i in range(M) if i != 40], [i for i in range(N) if i != 66]
    assert torch.equal(C[rm][:, rn], clean[rm][:, rn])


def test_no_contraction_no_rows():
    C = torch.full((5, 9), 3.0, device=DEV)
    pk = torch.empty(1024, dtype=torch.uint8, device=DEV)
    lac.fp8_gemm(pk, pk, 5, 9, 0, C=C, accumulate=True)
    assert (C == 3).all()
    assert not lac.fp8_gemm(pk, pk, 5, 9, 0, C=C).any()
    assert not lac.fp8_gemm(pk, pk, 5, 9, 0).any()
    assert lac.fp8_gemm(pk, pk, 0, 9, 4).shape == (0, 9)
    X = torch.empty(0, 40, device=DEV)
    p, _ = lac.fp8_pack(X)
    assert lac.fp8_unpack(p, 0, 40).shape == (0, 40)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("M, N, K", [(5, 37, 130), (70, 67, 260), (600, 261, 300), (40, 33, 9000)])
def test_products_write_their_rows_only_at_any_alignment(M, N, K, dt):
    A, B = data(M, K, "bf16", 8), data(N, K, "bf16", 9)
    pa, pb = lac.fp8_pack(A)[0], lac.fp8_pack(B)[0]
    buf = torch.full((M * N + 128,), 5.0, dtype=DT[dt], device=DEV)
    C = lac.fp8_gemm(pa, pb, M, N, K, C=buf[33:33 + M * N].view(M, N))
    assert torch.equal(C, lac.fp8_gemm(pa, pb, M, N, K, dtype=DT[dt]))
    assert (buf[:33] == 5).all() and (buf[33 + M * N:] == 5).all()
    out = torch.full((M * K + 64,), 5.0, dtype=DT[dt], device=DEV)
    lac.fp8_unpack(pa, M, K, X=out[31:31 + M * K].view(M, K))
    assert (out[:31] == 5).all() and (out[31 + M * K:] == 5).all()
    # packs stay inside their bytes, and sources of any offset give the same pack
    n = lac.fp8_pack_bytes(M, K)
    raw = torch.full((n + 64,), 0xA5, dtype=torch.uint8, device=DEV)
    src = torch.zeros(M * K + 5, dtype=torch.bfloat16, device=DEV)
    src[5:] = A.reshape(-1)
    lac.fp8_pack(src[5:].view(M, K), pk=raw[:n])
    assert (raw[n:] == 0xA5).all()
    assert torch.equal(lac.fp8_unpack(raw[:n], M, K), lac.fp8_unpack(pa, M, K))


def test_streams_repeats_and_graph():
    M, N, K = 257, 384, 4000
    A, B = data(M, K, "bf16", 10), data(N, K, "bf16", 11)
    pa, pb = lac.fp8_pack(A)[0], lac.fp8_pack(B)[0]
    C = lac.fp8_gemm(pa, pb, M, N, K, dtype=torch.float32)
    assert torch.equal(C, lac.fp8_gemm(pa, pb, M, N, K, dtype=torch.float32))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p2, _ = lac.fp8_pack(A, stream=s)
    C2 = lac.fp8_gemm(p2, pb, M, N, K, dtype=torch.float32, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(C, C2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p3, _ = lac.fp8_pack(A)
        C3 = lac.fp8_gemm(p3, pb, M, N, K)
    for turn in range(3):
        A.copy_(data(M, K, "bf16", 20 + turn))
        want = lac.fp8_gemm(lac.fp8_pack(A)[0], pb, M, N, K)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(C3, want)


def test_binding_refusals():
    pk = torch.empty(100, dtype=torch.uint8, device=DEV)
    A = torch.zeros(4, 8, device=DEV)
    for call, status in ((lambda: lac.fp8_gemm(pk, pk, 4, 4, 128), -5),
                         (lambda: lac.fp8_gemm(pk, pk, 4, 4, 128, accumulate=True), -1),
                         (lambda: lac.fp8_gemm(pk, pk, 4, 4, 0, C=A), -2),
                         (lambda: lac.fp8_pack(A.half()), -3), (lambda: lac.fp8_pack(A, rows=False), -1),
                         (lambda: lac.fp8_pack(A, pk=pk), -5), (lambda: lac.fp8_unpack(pk, 4, 8), -5),
                         (lambda: lac.fp8_pack(A.t()), -2)):
        with pytest.raises(lac.MaplError) as e:
            call()
        assert e.value.status == status
