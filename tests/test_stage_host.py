"""Pipeline-stage operators without a GPU: the oracle's definitions against
published values, loops and differences; the C ABI's refusals (each before
anything is enqueued) and its sizes; the binding's refusals."""
import ctypes

import numpy as np
import pytest
import torch

import learned_activation_compression_amd as lac
from learned_activation_compression_amd import stage as binding
from oracle import stage

OK, ENULL, ESHAPE, EDTYPE, EARG, EWS, EHIP = 0, -1, -2, -3, -4, -5, -6
F32, BF16 = lac.MAPL_F32, lac.MAPL_BF16
FAKE = ctypes.c_void_p(0x1000)  # never dereferenced
READY = OK if torch.cuda.is_available() else EHIP  # what a valid empty-gradient call returns


@pytest.fixture(scope="module")
def lib():
    return binding._stage_lib()


# ------------------------------------------------------------------ oracle --

@pytest.mark.parametrize("ctr, key, want", [
    ([0] * 4, [0] * 2, [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
    ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
    ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
     [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]),
])
def test_philox_known_answers(ctr, key, want):
    # the known answers published with the generator
    got = stage.philox4x32_10(np.array(ctr, dtype=np.uint64), key)
    assert [int(v) for v in got] == want


def test_keep_rate_and_independence():
    N, d, p = 512, 512, 0.3
    k = stage.keep(N, d, p, 12345678901234567, (1 << 40) + 5)
    t = stage.threshold(p)
    q = 1 - t / 65536
    # six standard deviations of a binomial
    assert abs(k.mean() - q) < 6 * np.sqrt(q * (1 - q) / k.size)
    assert np.array_equal(k[7:], stage.keep(N - 7, d, p, 12345678901234567, (1 << 40) + 12))  # rows are counters
    other = stage.keep(N, d, p, 12345678901234568, (1 << 40) + 5)
    both = (k & other).mean()
    assert abs(both - q * q) < 6 * np.sqrt(q * q * (1 - q * q) / k.size)


def test_dropout_edges():
    X = np.array([[np.inf, np.nan, 1.0, -2.0] * 8])
    assert np.array_equal(stage.dropout(X, 0.0, 1, 0), X, equal_nan=True)
    assert np.array_equal(stage.dropout(X, 1.0, 1, 0), np.zeros_like(X))
    k, y = stage.keep(1, 32, 0.5, 1, 0), stage.dropout(X, 0.5, 1, 0)
    assert np.all(y[~k] == 0) and np.array_equal(y[k], 2 * X[k], equal_nan=True)
    # the row counter wraps at 2^64
    assert np.array_equal(stage.keep(2, 8, 0.5, 1, (1 << 64) - 1)[1], stage.keep(1, 8, 0.5, 1, 0)[0])


@pytest.mark.parametrize("post, pre, G, p", [(1, 1, 1, 0.2), (1, 0, 3, 0.0), (0, 1, 6, 0.2), (0, 0, 0, 0.4),
                                             (1, 1, 6, 0.0), (1, 1, 0, 0.2)])
def test_norm_gradient_against_differences(post, pre, G, p):
    rng = np.random.default_rng(post + 2 * pre + 8 * G)
    N, d = 6, 11
    X, Y, gx, gh = (rng.standard_normal((N, d)) for _ in range(4))
    wp, wq = rng.standard_normal(d) if post else None, rng.standard_normal(d) if pre else None
    g = rng.standard_normal((G, d)) if G else None
    kw = dict(res_scale=0.7, eps=1e-3, p=p, seed=99, offset=7)

    def loss(X, Y, wp, g, wq):
        x, h = stage.norm(X, Y, wp, g, wq, **kw)
        return np.sum(x * gx) + (np.sum(h * gh) if pre else 0.0)

    x_out, _ = stage.norm(X, Y, wp, g, wq, **kw)
    got = stage.norm_bwd(gx, gh if pre else None, x_out, Y, wp, g, wq, **kw)
    args = dict(X=X, Y=Y, wp=wp, g=g, wq=wq)
    names = dict(X="gX", Y="gY", wp="g_w_post", g="g_gate", wq="g_w_pre")
    for k, v in args.items():
        if v is None:
            assert names[k] not in got
            continue
        num, step = np.empty_like(v), 1e-5
        for i in np.ndindex(*v.shape):
            hi, lo = v.copy(), v.copy()
            hi[i] += step
            lo[i] -= step
            num[i] = (loss(**{**args, k: hi}) - loss(**{**args, k: lo})) / (2 * step)
        # central differences: step^2 times third derivatives, and 2^-53 / step of the loss
        np.testing.assert_allclose(got[names[k]], num, rtol=1e-6, atol=1e-6)


def test_e4m3_against_the_library_cast():
    x = np.concatenate([np.linspace(-448, 448, 20001), np.random.default_rng(0).standard_normal(20000) * 0.05,
                        stage.GRID, (stage.GRID[1:] + stage.GRID[:-1]) / 2])
    want = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(stage.e4m3(x.astype(np.float32).astype(np.float64)), want)


def test_block_scales():
    X = np.zeros((2, 300))
    X[0, 0], X[0, 1] = 448.0, 2.0 ** -9
    X[0, 128] = 449.0
    X[1, 299] = 2.0 ** -140
    V = stage.round_blocks(X)
    assert V[0, 0] == 448 and V[0, 1] == 2.0 ** -9  # scale 1
    assert V[0, 128] == 448                        # scale 2: 224.5 is nearest to 224
    assert V[1, 299] == 0                          # below half of the smallest code at the smallest scale
    W = stage.round_blocks(np.tile(X, (1, 1)), square=True)
    assert np.array_equal(W.T, stage.round_blocks(np.ascontiguousarray(X.T), square=True))


# --------------------------------------------------------------------- ABI --

def test_library_exports_the_stage_symbols(lib):
    names = binding.stage_symbols()
    assert set(names) == set(binding._STAGE_SIGS) and len(names) == 9
    for n in names:
        assert hasattr(lib, n), n
        assert callable(getattr(lac, n))


def _dropout(lib, **kw):
    a = dict(X=FAKE, Y=FAKE, p=0.1, seed=1, offset=0, N=0, d=64, dt=BF16)
    a.update(kw)
    return lib.stage_dropout(*a.values(), None)


def test_dropout_refusals(lib):
    assert _dropout(lib) == OK and _dropout(lib, X=None, Y=None) == OK  # no rows
    assert _dropout(lib, p=0.0) == OK and _dropout(lib, p=1.0) == OK
    for p in (-0.1, 1.0000001, float("nan"), float("inf")):
        assert _dropout(lib, p=p) == EARG
    assert _dropout(lib, dt=5) == EDTYPE
    for bad in (dict(N=-1), dict(d=0), dict(N=2 ** 31), dict(d=2 ** 31 - 7), dict(N=2 ** 30, d=2 ** 7)):
        assert _dropout(lib, **bad) == ESHAPE, bad
    assert _dropout(lib, N=1, X=None) == ENULL and _dropout(lib, N=1, Y=None) == ENULL
    assert _dropout(lib, N=1, X=ctypes.c_void_p(0x1001)) == EARG
    assert _dropout(lib, N=1, dt=F32, X=ctypes.c_void_p(0x1002)) == EARG


def _norm(lib, **kw):
    a = dict(X=FAKE, Y=FAKE, w_post=FAKE, gate=FAKE, w_pre=FAKE, X_out=FAKE, H=FAKE, res_scale=1.0, eps=1e-5, p=0.1,
             seed=1, offset=0, N=0, d=64, G=1, dt=BF16)
    a.update(kw)
    return lib.stage_norm(*a.values(), None)


def _norm_bwd(lib, **kw):
    a = dict(gX_out=FAKE, gH=FAKE, X_out=FAKE, Y=FAKE, w_post=FAKE, gate=FAKE, w_pre=FAKE, gX=FAKE, gY=FAKE,
             g_w_post=FAKE, g_gate=FAKE, g_w_pre=FAKE, accumulate=1, res_scale=1.0, eps=1e-5, p=0.1, seed=1, offset=0,
             N=0, d=64, G=1, dt=BF16, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return lib.stage_norm_bwd(*a.values(), None)


@pytest.mark.parametrize("call", [_norm, _norm_bwd])
def test_norm_common_refusals(lib, call):
    assert call(lib) == OK  # no rows (the gradient accumulates)
    assert call(lib, dt=9) == EDTYPE
    for bad in (dict(N=-1), dict(N=2 ** 31), dict(d=0), dict(d=8193), dict(G=-1), dict(N=10, G=3), dict(N=2, G=4)):
        assert call(lib, **bad) == ESHAPE, bad
    for bad in (dict(eps=0.0), dict(eps=1e-39), dict(eps=-1.0), dict(eps=float("inf")), dict(eps=float("nan")), dict(p=1.5),
                dict(p=float("nan")), dict(res_scale=float("inf")), dict(gate=None), dict(G=0),
                dict(N=4, Y=None), dict(N=4, Y=None, p=0.0), dict(N=4, Y=None, p=0.0, w_post=None)):
        assert call(lib, **bad) == EARG, bad
    none = dict(Y=None, p=0.0, w_post=None, gate=None, G=0)
    assert call(lib, **none) == OK
    assert call(lib, **{**none, "p": 0.1}, N=4) == EARG


def test_norm_refusals(lib):
    assert _norm(lib, N=4, X=None) == ENULL
    assert _norm(lib, N=4, X_out=None, H=None, w_pre=None) == ENULL
    assert _norm(lib, N=4, w_pre=None) == ENULL
    assert _norm(lib, N=4, H=None) == EARG       # a weight without its output
    assert _norm(lib, N=4, gate=ctypes.c_void_p(0x1001)) == EARG


def test_norm_bwd_refusals(lib):
    assert _norm_bwd(lib, accumulate=2) == EARG
    assert _norm_bwd(lib, accumulate=0) == READY  # zero gradients are written
    for missing in ("g_w_post", "g_gate"):
        assert _norm_bwd(lib, **{missing: None}) == ENULL, missing
    for missing in ("g_w_pre", "w_pre", "gX", "gY", "X_out", "ws"):
        assert _norm_bwd(lib, N=4, **{missing: None}) == ENULL, missing
    assert _norm_bwd(lib, N=4, gX_out=None, gH=None) == ENULL
    assert _norm_bwd(lib, N=4, ws=ctypes.c_void_p(0x1008)) == EARG
    assert _norm_bwd(lib, N=4, g_gate=ctypes.c_void_p(0x1002)) == EARG
    assert _norm_bwd(lib, N=4, ws_bytes=lib.stage_norm_bwd_workspace_bytes(4, 64, 1) - 1) == EWS
    assert lib.stage_norm_bwd_workspace_bytes(0, 64, 1) == 0
    assert lib.stage_norm_bwd_workspace_bytes(10, 64, 3) == 0
    assert lib.stage_norm_bwd_workspace_bytes(2 ** 31 - 1, 8192, 0) > 0


def test_fp8_sizes(lib):
    # 32-row x 128-column units of 4 KB, an exponent per row (rows to 256) and 128 columns, 256 bytes of slack
    assert lib.fp8_pack_bytes(1000, 1000) == 32 * 8 * 4096 + 8 * 1024 + 256
    assert lib.fp8_pack_bytes(1, 1) == 4096 + 256 + 256
    assert lib.fp8_pack_bytes(-1, 4) == 0 and lib.fp8_pack_bytes(2 ** 30 + 1, 1) == 0
    assert lib.fp8_pack_bytes(2 ** 30, 2 ** 7) == 0
    assert lib.fp8_gemm_workspace_bytes(0, 8, 8) == 0 and lib.fp8_gemm_workspace_bytes(8, 8, -8) == 0


def test_fp8_pack_refusals(lib):
    def pack(**kw):
        a = dict(X=FAKE, pk=FAKE, pk_bytes=1 << 40, pkT=FAKE, pkT_bytes=1 << 40, square=0, R=4, C=4, dt=BF16)
        a.update(kw)
        return lib.fp8_pack(*a.values(), None)
    assert pack(R=0) == OK and pack(C=0, X=None, pk=None, pkT=None) == OK
    assert pack(dt=3) == EDTYPE and pack(R=-1) == ESHAPE and pack(R=2 ** 30, C=2 ** 10) == ESHAPE
    assert pack(square=2) == EARG and pack(X=None) == ENULL and pack(pk=None, pkT=None) == ENULL
    assert pack(pk=ctypes.c_void_p(0x1008)) == EARG and pack(pkT=ctypes.c_void_p(0x1008)) == EARG
    assert pack(pk_bytes=lib.fp8_pack_bytes(4, 4) - 1) == EWS
    assert pack(R=4, C=400, pkT_bytes=lib.fp8_pack_bytes(4, 400)) == EWS  # the transpose has its own size
    assert pack(X=ctypes.c_void_p(0x1001)) == EARG


def test_fp8_unpack_and_gemm_refusals(lib):
    def unpack(**kw):
        a = dict(pk=FAKE, pk_bytes=1 << 40, X=FAKE, rows=4, cols=4, dt=BF16)
        a.update(kw)
        return lib.fp8_unpack(*a.values(), None)
    assert unpack(rows=0) == OK and unpack(dt=2) == EDTYPE and unpack(cols=-1) == ESHAPE
    assert unpack(pk=None) == ENULL and unpack(X=None) == ENULL and unpack(pk_bytes=100) == EWS

    def gemm(**kw):
        a = dict(A=FAKE, A_bytes=1 << 40, B=FAKE, B_bytes=1 << 40, C=FAKE, acc=0, M=64, N=64, K=64, dt=BF16, ws=FAKE,
                 ws_bytes=1 << 40)
        a.update(kw)
        return lib.fp8_gemm(*a.values(), None)
    assert gemm(M=0) == OK and gemm(N=0) == OK and gemm(dt=-1) == EDTYPE
    for bad in (dict(M=-1), dict(K=-1), dict(N=2 ** 31), dict(M=2 ** 30, N=2 ** 7), dict(M=2 ** 30, K=2 ** 7)):
        assert gemm(**bad) == ESHAPE, bad
    assert gemm(acc=1) == EARG and gemm(acc=2, dt=F32) == EARG  # bf16 does not accumulate
    assert gemm(A=None) == ENULL and gemm(B=None) == ENULL and gemm(C=None) == ENULL
    assert gemm(A=ctypes.c_void_p(0x1004)) == EARG and gemm(C=ctypes.c_void_p(0x1001)) == EARG
    assert gemm(A_bytes=10) == EWS and gemm(B_bytes=10) == EWS


def test_binding_refuses_host_tensors_and_bad_scalars():
    X = torch.zeros(4, 8)
    for call in (lambda: lac.stage_dropout(X, 0.1, 1), lambda: lac.stage_norm(X), lambda: lac.stage_norm_bwd(X),
                 lambda: lac.fp8_pack(X), lambda: lac.stage_norm_bwd()):
        with pytest.raises(lac.MaplError) as e:
            call()
        assert e.value.status == -1
    with pytest.raises(lac.MaplError):
        lac.stage_dropout(torch.zeros(4), 0.1, 1)
    with pytest.raises(lac.MaplError):
        binding._u(-1, "seed")
    with pytest.raises(lac.MaplError):
        binding._u(1 << 64, "seed")
