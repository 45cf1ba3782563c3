"""Operators between a stage's boundary and its loss without a GPU: the oracle's
definitions against loops and differences; the C ABI's refusals (each before
anything is enqueued) and its sizes; the binding's refusals."""
import ctypes

import numpy as np
import pytest
import torch

import learned_activation_compression_amd as lac
from learned_activation_compression_amd import block as binding
from oracle import block

OK, ENULL, ESHAPE, EDTYPE, EARG, EWS, EHIP = 0, -1, -2, -3, -4, -5, -6
F32, BF16 = lac.MAPL_F32, lac.MAPL_BF16
FAKE = ctypes.c_void_p(0x1000)  # never dereferenced
ODD = ctypes.c_void_p(0x1001)
no_device = pytest.mark.skipif(torch.cuda.is_available(), reason="a device is present: valid calls would launch kernels")


@pytest.fixture(scope="module")
def lib():
    return binding._block_lib()


def test_library_exports_the_block_symbols(lib):
    names = binding.block_symbols()
    assert set(names) == set(binding._BLOCK_SIGS) == set(binding.__all__)
    for n in names:
        assert hasattr(lib, n), n
        assert callable(getattr(lac, n)) and n in lac.__all__


def differences(loss, args, name, step=1e-5):
    num = np.empty_like(args[name])
    for i in np.ndindex(*num.shape):
        hi, lo = args[name].copy(), args[name].copy()
        hi[i] += step
        lo[i] -= step
        num[i] = (loss(**{**args, name: hi}) - loss(**{**args, name: lo})) / (2 * step)
    return num


# --------------------------------------------------------------- attention --

@pytest.mark.parametrize("lens, Hq, Hkv, D", [([3, 4], 2, 1, 3), ([1, 5, 2], 2, 2, 2), ([6], 4, 2, 2)])
def test_attention_gradient_against_differences(lens, Hq, Hkv, D):
    rng = np.random.default_rng(Hq + D)
    N, cu, c = sum(lens), np.cumsum([0, *lens]), 0.7
    a = dict(q=rng.standard_normal((N, Hq, D)), k=rng.standard_normal((N, Hkv, D)), v=rng.standard_normal((N, Hkv, D)))
    go = rng.standard_normal((N, Hq, D))
    o, lse, _, _ = block.attn(**a, cu=cu, scale=c)
    g, _ = block.attn_bwd(go, **a, o=o, lse=lse, cu=cu, scale=c)
    for n in a:
        num = differences(lambda **x: np.sum(block.attn(**x, cu=cu, scale=c)[0] * go), a, n)
        # central differences: step^2 times third derivatives, and 2^-53 / step of the loss
        np.testing.assert_allclose(g["g" + n], num, rtol=1e-6, atol=1e-6)


def test_attention_of_one_row_and_of_equal_scores():
    v = np.arange(12.0).reshape(4, 1, 3)
    o, lse, _, _ = block.attn(np.zeros((4, 1, 3)), np.ones((4, 1, 3)), v, [0, 1, 4], 1.0)
    assert np.allclose(o[0], v[0]) and np.allclose(o[3, 0], v[1:4, 0].mean(0)) and np.allclose(lse[0], np.log([1, 1, 2, 3]))


def _attn(lib, **kw):
    a = dict(Q=FAKE, K=FAKE, V=FAKE, cu=FAKE, O=FAKE, lse=FAKE, scale=0.1, S=1, N=0, Hq=4, Hkv=2, D=64, ldq=256, ldk=128,
             ldv=128, ldo=256, dt=BF16)
    a.update(kw)
    return lib.stage_attn(*a.values(), None)


def _attn_bwd(lib, **kw):
    a = dict(gO=FAKE, Q=FAKE, K=FAKE, V=FAKE, O=FAKE, lse=FAKE, cu=FAKE, gQ=FAKE, gK=FAKE, gV=FAKE, scale=0.1, S=1, N=0,
             Hq=4, Hkv=2, D=64, ldgo=256, ldq=256, ldk=128, ldv=128, ldo=256, ldgq=256, ldgk=128, ldgv=128, dt=BF16,
             ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return lib.stage_attn_bwd(*a.values(), None)


@pytest.mark.parametrize("call", [_attn, _attn_bwd])
def test_attention_refusals(lib, call):
    assert call(lib) == OK and call(lib, N=5, S=0) == OK  # no rows, no sequences
    assert call(lib, Q=None, K=None, cu=None) == OK
    assert call(lib, dt=7) == EDTYPE
    for bad in (dict(N=-1), dict(S=-1), dict(S=2 ** 31 - 1), dict(Hq=0), dict(Hkv=0), dict(Hq=3), dict(Hq=1), dict(D=0),
                dict(D=129), dict(N=2 ** 28 + 1), dict(Hq=1 << 17, Hkv=1 << 17), dict(ldq=255), dict(ldk=127), dict(ldv=-128),
                dict(ldo=2 ** 22 + 1)):
        assert call(lib, **bad) == ESHAPE, bad
    for s in (0.0, -0.1, 2.0 ** -65, 2.0 ** 65, float("inf"), float("nan")):
        assert call(lib, scale=s) == EARG
    for n in ("Q", "K", "V", "cu", "O", "lse"):
        assert call(lib, N=4, **{n: None}) == ENULL, n
        assert call(lib, N=4, **{n: ODD}) == EARG, n
    assert call(lib, N=4, dt=F32, K=ctypes.c_void_p(0x1002)) == EARG


def test_attention_backward_refusals(lib):
    for n in ("gO", "gQ", "gK", "gV", "ws"):
        assert _attn_bwd(lib, N=4, **{n: None}) == ENULL, n
        assert _attn_bwd(lib, N=4, **{n: ODD}) == EARG, n
    for n, ld in (("ldgo", 255), ("ldgq", 255), ("ldgk", 127), ("ldgv", 2 ** 22 + 1)):
        assert _attn_bwd(lib, N=4, **{n: ld}) == ESHAPE, n
    assert _attn_bwd(lib, N=4, ws=ctypes.c_void_p(0x1008)) == EARG
    need = lib.stage_attn_bwd_workspace_bytes(4, 4, 2, 64)
    assert need >= 2 * 4 * 4 * 4 and _attn_bwd(lib, N=4, ws_bytes=need - 1) == EWS
    assert lib.stage_attn_bwd_workspace_bytes(-1, 4, 2, 64) == 0 and lib.stage_attn_bwd_workspace_bytes(4, 4, 3, 64) == 0


@no_device
@pytest.mark.parametrize("call", [_attn, _attn_bwd])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_attention_takes_what_it_documents(lib, call, dt):
    for kw in (dict(N=1), dict(N=2 ** 28), dict(N=7, D=1), dict(N=7, D=128, ldq=512, ldk=256, ldv=2 ** 22, ldo=512,
                                                               **(dict(ldgo=512, ldgq=512, ldgk=256, ldgv=256)
                                                                  if call is _attn_bwd else {}))):
        assert call(lib, dt=dt, **kw) == EHIP, kw  # the device set-up's error


def test_binding_refuses_host_tensors():
    q, cu = torch.zeros(4, 2, 8), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: lac.stage_attn(q, q, q, cu), lambda: lac.stage_attn(q, q, q, None),
                 lambda: lac.stage_attn_bwd(q, q, q, q, q, q, cu), lambda: lac.stage_attn(q, q, q, 3)):
        with pytest.raises(lac.MaplError) as e:
            call()
        assert e.value.status == -1


# -------------------------------------------------------------------- loss --

@pytest.mark.parametrize("T, w_ce, w_kd", [(1.0, 1.0, 0.0), (2.0, 0.3, 4.0), (1.0, 0.0, 1.0), (0.5, 1.0, 1.0)])
def test_loss_gradient_against_differences(T, w_ce, w_kd):
    rng = np.random.default_rng(7)
    N, V, K = 5, 9, 4
    Z, t, g = rng.standard_normal((N, V)), rng.standard_normal((N, K)), rng.standard_normal(N)
    y, ids = np.array([0, -1, 8, 3, 9]), rng.integers(0, V, (N, K))
    ids[1], ids[2, 1], ids[3] = -1, 40, [2, 2, 3, 2]  # a row of none, an id too large, one id three times
    t[0, 0] = -np.inf
    got, _ = block.distill_bwd(g, Z, y, ids, t, T, w_ce, w_kd)
    num = differences(lambda Z: np.sum(g * block.distill(Z, y, ids, t, T, w_ce, w_kd)[0]), dict(Z=Z), "Z")
    np.testing.assert_allclose(got, num, rtol=1e-6, atol=1e-6)
    assert np.all(got[1] == 0)


def test_loss_of_equal_logits_and_of_the_teacher_itself():
    Z, ids = np.zeros((2, 8)), np.array([[0, 1], [5, 6]])
    loss, stats, _ = block.distill(Z, np.array([3, -1]), ids, np.zeros((2, 2)), 1.0, 1.0, 0.0)
    assert np.allclose(loss, [np.log(8), 0]) and np.allclose(stats, np.log(8))
    # a teacher that gives all entries and agrees: no divergence and no gradient
    Z = np.random.default_rng(0).standard_normal((1, 8))
    args = (None, np.arange(8)[None], Z.copy(), 2.0, 1.0, 1.0)
    assert np.allclose(block.distill(Z, *args)[0], 0) and np.allclose(block.distill_bwd(np.ones(1), Z, *args)[0], 0)


def _distill(lib, **kw):
    a = dict(Z=FAKE, labels=FAKE, t_ids=FAKE, t_logits=FAKE, loss=FAKE, stats=FAKE, T=2.0, w_ce=1.0, w_kd=1.0, N=0, V=100,
             K=8, dt=BF16, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return lib.stage_distill(*a.values(), None)


def _distill_bwd(lib, **kw):
    a = dict(gloss=FAKE, Z=FAKE, stats=FAKE, labels=FAKE, t_ids=FAKE, t_logits=FAKE, gZ=FAKE, T=2.0, w_ce=1.0, w_kd=1.0,
             N=0, V=100, K=8, dt=BF16)
    a.update(kw)
    return lib.stage_distill_bwd(*a.values(), None)


@pytest.mark.parametrize("call", [_distill, _distill_bwd])
def test_loss_refusals(lib, call):
    assert call(lib) == OK and call(lib, Z=None, stats=None) == OK  # no rows
    assert call(lib, dt=2) == EDTYPE
    for bad in (dict(N=-1), dict(N=2 ** 23 + 1), dict(V=0), dict(V=2 ** 27 + 1), dict(K=-1), dict(K=1025),
                dict(N=2 ** 20, V=2 ** 17)):
        assert call(lib, **bad) == ESHAPE, bad
    for bad in (dict(T=0.0), dict(T=-1.0), dict(T=float("inf")), dict(T=float("nan")), dict(T=1e-40),
                dict(w_ce=float("nan")), dict(w_kd=float("inf"))):
        assert call(lib, **bad) == EARG, bad
    for n in ("Z", "stats", "t_ids", "t_logits"):
        assert call(lib, N=4, **{n: None}) == ENULL, n
        assert call(lib, N=4, **{n: ODD}) == EARG, n
    assert call(lib, N=4, labels=ODD) == EARG


def test_loss_refusals_of_one_direction(lib):
    assert _distill(lib, N=4, loss=None) == ENULL and _distill(lib, N=4, loss=ODD) == EARG
    for n in ("gloss", "gZ"):
        assert _distill_bwd(lib, N=4, **{n: None}) == ENULL and _distill_bwd(lib, N=4, **{n: ODD}) == EARG
    need = lib.stage_distill_workspace_bytes(4, 131072)
    assert need > 0 and lib.stage_distill_workspace_bytes(4, 100) == 0 and lib.stage_distill_workspace_bytes(5000, 32000) == 0
    assert lib.stage_distill_workspace_bytes(0, 100) == 0 and lib.stage_distill_workspace_bytes(4, -1) == 0
    big = dict(N=4, V=131072)
    assert _distill(lib, **big, ws=None) == ENULL and _distill(lib, **big, ws=ctypes.c_void_p(0x1008)) == EARG
    assert _distill(lib, **big, ws_bytes=need - 1) == EWS


@no_device
@pytest.mark.parametrize("call", [_distill, _distill_bwd])
def test_loss_takes_what_it_documents(lib, call):
    for kw in (dict(N=1), dict(N=2 ** 23, V=1), dict(N=1, V=2 ** 27), dict(N=3, K=0, t_ids=None, t_logits=None),
               dict(N=3, labels=None), dict(N=3, K=1024), dict(N=3, dt=F32)):
        assert call(lib, **kw) == EHIP, kw


# -------------------------------------------------------------- block edge --

def _norm_pack(lib, **kw):
    a = dict(X=FAKE, Y=FAKE, w_post=FAKE, gate=FAKE, w_pre=FAKE, X_out=FAKE, H=FAKE, pk=FAKE, pk_bytes=1 << 40,
             res_scale=1.0, eps=1e-5, p=0.1, seed=1, offset=0, N=0, d=64, G=1, dt=BF16)
    a.update(kw)
    return lib.stage_norm_pack(*a.values(), None)


def test_norm_pack_refusals(lib):
    assert _norm_pack(lib) == OK and _norm_pack(lib, X=None, pk=None) == OK
    assert _norm_pack(lib, dt=9) == EDTYPE
    for bad in (dict(N=-1), dict(N=2 ** 27 + 1), dict(N=2 ** 24, d=8192), dict(d=0), dict(d=8193), dict(G=-1),
                dict(N=10, G=3), dict(N=2, G=4)):
        assert _norm_pack(lib, **bad) == ESHAPE, bad
    for bad in (dict(eps=0.0), dict(eps=float("nan")), dict(p=1.5), dict(res_scale=float("inf")), dict(gate=None), dict(G=0),
                dict(N=4, Y=None), dict(N=4, X=ODD), dict(N=4, H=ODD), dict(N=4, pk=ctypes.c_void_p(0x1008))):
        assert _norm_pack(lib, **bad) == EARG, bad
    for n in ("X", "w_pre", "pk"):
        assert _norm_pack(lib, N=4, **{n: None}) == ENULL, n
    assert _norm_pack(lib, N=4, pk_bytes=lib.fp8_pack_bytes(4, 64) - 1) == EWS


@no_device
def test_norm_pack_takes_what_it_documents(lib):
    none = dict(Y=None, p=0.0, w_post=None, gate=None, G=0)
    for kw in (dict(N=4), dict(N=4, X_out=None, H=None), dict(N=4, **none), dict(N=2 ** 23, d=8192), dict(N=5, d=7, dt=F32)):
        assert _norm_pack(lib, **kw) == EHIP, kw


def test_binding_refuses_host_tensors_of_the_other_operators():
    x = torch.zeros(4, 8)
    for call in (lambda: lac.stage_norm_pack(x, w_pre=x[0]), lambda: lac.stage_distill(x),
                 lambda: lac.stage_distill_bwd(x[:, 0], x, x[:, :2])):
        with pytest.raises(lac.MaplError) as e:
            call()
        assert e.value.status == -1
