"""Dropout and the block edge on the GPU against the float64 oracle.

Tolerances.  An output is rounded once, by at most half a step of its type
(eps / 2 of its value).  Before that everything is fp32: the sums of squares
and dot products add d terms in at most d / 8 + 16 additions on any path, and a
handful of products and one reciprocal square root follow, so an error is at
most STEPS(d) half steps of fp32 of the size of the sum, where every term
counts by its absolute value (the oracle's size = True).  Sums over rows add
N terms more."""
import numpy as np
import pytest
import torch

import learned_activation_compression_amd as lac
from oracle import stage

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
F32_HALF = torch.finfo(torch.float32).eps / 2


def n64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def steps(d):
    return d / 8 + 32


def near(got, ref, size, out_dtype, count, what):
    got = n64(got)
    bound = torch.finfo(out_dtype).eps / 2 * np.abs(ref) + count * F32_HALF * size + torch.finfo(torch.float32).tiny
    # the rounding of the output is half a step of the rounded fp32 value, not of the reference
    bound = bound * (1 + 2.0 ** -7)
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} against {ref[bad][0]} (bound {bound[bad][0]:.3e})")


def rows(rng, N, d, dt, scale=1.0):
    return torch.from_numpy((rng.standard_normal((N, d)) * np.exp(0.5 * rng.standard_normal(d)) * scale)
                            .astype(np.float32)).to(DT[dt]).to(DEV)


def vec(rng, shape, dt, mean=0.0):
    return torch.from_numpy((mean + 0.3 * rng.standard_normal(shape)).astype(np.float32)).to(DT[dt]).to(DEV)


# ----------------------------------------------------------------- dropout --

@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N, d", [(1, 1), (3, 7), (5, 8), (129, 9), (7, 1003), (64, 1024), (1, 100001), (3001, 16)])
def test_dropout(N, d, dt):
    rng = np.random.default_rng(N + d)
    X = rows(rng, N, d, dt)
    seed, off = 0xFEDCBA9876543210, (1 << 33) - 2  # the row counter's low word wraps inside
    for p in (0.1, 0.5):
        Y = lac.stage_dropout(X, p, seed, off)
        k = stage.keep(N, d, p, seed, off)
        got = n64(Y)
        assert np.array_equal(got[~k], np.zeros((~k).sum()))
        ref = stage.dropout(n64(X), p, seed, off)
        near(Y, ref, np.abs(ref), DT[dt], 3, "dropout")
    assert torch.equal(lac.stage_dropout(X, 0.0, seed, off), X)
    assert not lac.stage_dropout(X, 1.0, seed, off).any()


def test_dropout_of_values_that_are_not_finite_and_in_place():
    X = torch.tensor([float("inf"), float("nan"), -float("inf"), 1.0] * 64, device=DEV).reshape(4, 64)
    k = torch.from_numpy(stage.keep(4, 64, 0.5, 3, 0)).to(DEV)
    Y = lac.stage_dropout(X, 0.5, 3)
    assert (Y[~k] == 0).all()
    assert torch.equal(Y[k].nan_to_num(nan=7.0), (X[k] * 2).nan_to_num(nan=7.0))
    Z = X.clone()
    assert lac.stage_dropout(Z, 0.5, 3, Y=Z) is Z and torch.equal(Z.nan_to_num(nan=7.0), Y.nan_to_num(nan=7.0))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_dropout_writes_its_rows_only_at_any_alignment(dt):
    d, N = 37, 11
    buf = torch.full((N * d + 64,), 5.0, dtype=DT[dt], device=DEV)
    src = torch.randn(N * d + 3, device=DEV).to(DT[dt])
    X, Y = src[3:].view(N, d), buf[17:17 + N * d].view(N, d)
    lac.stage_dropout(X, 0.25, 5, 6, Y=Y)
    assert torch.equal(Y, lac.stage_dropout(X.clone(), 0.25, 5, 6))
    assert (buf[:17] == 5).all() and (buf[17 + N * d:] == 5).all()


# -------------------------------------------------------------- block edge --

WIDTHS = [1, 5, 16, 64, 65, 128, 200, 256, 500, 512, 1000, 1024, 1536, 2047, 2048, 4096, 5000, 8192]


def edge_inputs(N, d, dt, post, pre, G, seed=0):
    rng = np.random.default_rng(1000 * N + d + seed)
    a = dict(X=rows(rng, N, d, dt), Y=rows(rng, N, d, dt, 0.5),
             w_post=vec(rng, d, dt, 1.0) if post else None, gate=vec(rng, (G, d), dt, 0.3) if G else None,
             w_pre=vec(rng, d, dt, 1.0) if pre else None)
    if N > 2:
        a["Y"][1] = 0  # a padding token
    return a, rng


def check_edge(N, d, dt, post, pre, G, p, offset=(1 << 32) - 1):
    a, rng = edge_inputs(N, d, dt, post, pre, G)
    kw = dict(res_scale=0.7, eps=1e-5, p=p, seed=77 << 32 | 5, offset=offset)
    x, h = lac.stage_norm(**a, **kw)
    b = {k: n64(v) for k, v in a.items()}
    xr, hr = stage.norm(b["X"], b["Y"], b["w_post"], b["gate"], b["w_pre"], **kw)
    ab = {k: None if v is None else np.abs(v) for k, v in b.items()}
    size, _ = stage.norm(ab["X"], ab["Y"], ab["w_post"], ab["gate"], None, **kw)
    near(x, xr, size, DT[dt], steps(d), "X_out")
    if pre:
        r = 1 / np.sqrt((xr ** 2).mean(1, keepdims=True) + 1e-5)
        # an error of a column moves its own output, and all errors of the row move the norm
        row = np.sqrt((size ** 2).mean(1, keepdims=True)) * r
        near(h, hr, ab["w_pre"] * r * size + np.abs(hr) * (1 + row), DT[dt], steps(d), "H")
    else:
        assert h is None

    gx, gh = rows(rng, N, d, dt, 1e-3), rows(rng, N, d, dt, 1e-3) if pre else None
    grads = lac.stage_norm_bwd(gx, gh, x, a["Y"], a["w_post"], a["gate"], a["w_pre"], **kw)
    args = (n64(gx), n64(gh), n64(x), b["Y"], b["w_post"], b["gate"], b["w_pre"])
    ref = stage.norm_bwd(*args, **kw)
    big = stage.norm_bwd(*args, **kw, size=True)
    for name, got in zip(("gX", "gY", "g_w_post", "g_gate", "g_w_pre"), grads):
        if name not in ref:
            assert got is None, name
            continue
        sums = name not in ("gX", "gY")
        near(got, ref[name], big[name], torch.float32 if sums else DT[dt], 4 * steps(d) + (N if sums else 0), name)
    return a, kw, (gx, gh, x), grads


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", WIDTHS)
def test_edge_over_widths(d, dt):
    check_edge(37, d, dt, True, True, 1, 0.2)


@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 63, 513, 2050])
@pytest.mark.parametrize("d", [96, 1024])
def test_edge_over_rows(N, d):
    check_edge(N, d, "bf16", True, True, 1, 0.0)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("post, pre, G, p", [
    (0, 0, 0, 0.0), (0, 0, 0, 0.5), (1, 0, 0, 0.1), (0, 1, 0, 0.1), (0, 1, 1, 0.1), (1, 0, 12, 0.1), (1, 1, 12, 0.0),
    (1, 1, 1200, 0.1), (1, 1, 600, 0.0), (0, 0, 1200, 0.0), (1, 1, 400, 0.3)])
def test_edge_parts_and_gates(post, pre, G, p, dt):
    # 1200 rows: a gate per row and per two rows (written row by row), per 3 rows and per 100 (joined from partial sums)
    check_edge(1200, 200, dt, post, pre, G, p)


@pytest.mark.parametrize("d", [40, 2048])
def test_edge_with_a_gate_per_token(d):
    check_edge(1111, d, "bf16", True, True, 1111, 0.1)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_norm_in_front_of_the_first_block(dt):
    rng = np.random.default_rng(4)
    N, d = 33, 1000
    X, w, gh = rows(rng, N, d, dt), vec(rng, d, dt, 1.0), rows(rng, N, d, dt)
    x, h = lac.stage_norm(X, w_pre=w, store_x=False)
    assert x is None
    xr, hr = stage.norm(n64(X), w_pre=n64(w))
    near(h, hr, 2 * np.abs(hr), DT[dt], steps(d), "H")
    gX, gY, gp, gg, gw = lac.stage_norm_bwd(None, gh, X, w_pre=w)
    assert gY is None and gp is None and gg is None
    args = (None, n64(gh), n64(X), None, None, None, n64(w), 1.0, 1e-5, 0.0, 0, 0)
    ref, big = stage.norm_bwd(*args), stage.norm_bwd(*args, size=True)
    near(gX, ref["gX"], big["gX"], DT[dt], 4 * steps(d), "gX")
    near(gw, ref["g_w_pre"], big["g_w_pre"], torch.float32, 4 * steps(d) + N, "g_w_pre")


def test_gradients_accumulate_repeat_and_take_given_buffers():
    a, kw, (gx, gh, x), first = check_edge(600, 1024, "bf16", True, True, 4, 0.1)
    call = lambda **k: lac.stage_norm_bwd(gx, gh, x, a["Y"], a["w_post"], a["gate"], a["w_pre"], **kw, **k)  # noqa: E731
    again = call()
    for s, t in zip(first, again):
        assert torch.equal(s, t)  # bitwise repeatable
    sums = [torch.full_like(t, 0.5) for t in first[2:]]
    out = call(g_w_post=sums[0], g_gate=sums[1], g_w_pre=sums[2], accumulate=True)
    for s, t in zip(out[2:], first[2:]):
        assert torch.equal(s, 0.5 + t)
    # documented aliases: gX over gX_out, gY over Y; the forward's X_out over X
    y, g = a["Y"].clone(), gx.clone()
    out = lac.stage_norm_bwd(g, gh, x, y, a["w_post"], a["gate"], a["w_pre"], **kw, gX=g, gY=y)
    assert torch.equal(out[0], first[0]) and torch.equal(out[1], first[1])
    x2 = a["X"].clone()
    x3, h3 = lac.stage_norm(x2, a["Y"], a["w_post"], a["gate"], a["w_pre"], **kw, X_out=x2)
    assert torch.equal(x3, x) and x3 is x2
    # gate per token accumulates in its own kernel path
    G = 600
    ga = torch.randn(G, 1024, device=DEV).bfloat16()
    r = lac.stage_norm_bwd(gx, gh, x, a["Y"], a["w_post"], ga, a["w_pre"], **kw)
    pre = [torch.full_like(t, 0.25) for t in r[2:]]
    r2 = lac.stage_norm_bwd(gx, gh, x, a["Y"], a["w_post"], ga, a["w_pre"], **kw, g_w_post=pre[0], g_gate=pre[1],
                            g_w_pre=pre[2], accumulate=True)
    for s, t in zip(r2[2:], r[2:]):
        assert torch.equal(s, 0.25 + t)


def test_rows_that_are_not_finite_stay_rows():
    a, rng = edge_inputs(9, 500, "f32", True, True, 1)
    gx, gh = rows(rng, 9, 500, "f32"), rows(rng, 9, 500, "f32")
    clean_x, clean_h = lac.stage_norm(**a)
    clean = lac.stage_norm_bwd(gx, gh, clean_x, a["Y"], a["w_post"], a["gate"], a["w_pre"])
    a["Y"][3, 17] = float("nan")
    a["X"][6, 2] = float("inf")
    x, h = lac.stage_norm(**a)
    ok = [0, 1, 2, 4, 5, 7, 8]
    assert torch.equal(x[ok], clean_x[ok]) and torch.equal(h[ok], clean_h[ok])
    assert x[3].isnan().all() and h[3].isnan().all() and h[6, 2].isnan()
    g = lac.stage_norm_bwd(gx, gh, x, a["Y"], a["w_post"], a["gate"], a["w_pre"])
    assert torch.equal(g[0][ok], clean[0][ok]) and torch.equal(g[1][ok], clean[1][ok])
    # dropped places may hold anything
    k = torch.from_numpy(stage.keep(9, 500, 0.5, 8, 0)).to(DEV)
    y = torch.where(k, clean_x, torch.full_like(clean_x, float("nan")))
    x1, h1 = lac.stage_norm(clean_x, y, a["w_post"], p=0.5, seed=8)
    x2, h2 = lac.stage_norm(clean_x, torch.where(k, clean_x, torch.zeros_like(clean_x)), a["w_post"], p=0.5, seed=8)
    assert torch.equal(x1, x2)


def test_no_rows():
    for dt in (torch.bfloat16, torch.float32):
        X = torch.empty(0, 64, dtype=dt, device=DEV)
        w = torch.ones(64, dtype=dt, device=DEV)
        x, h = lac.stage_norm(X, X, w, None, w)
        assert x.shape == (0, 64) and h.shape == (0, 64) and lac.stage_dropout(X, 0.5, 1).shape == (0, 64)
        g = lac.stage_norm_bwd(X, X, X, X, w, w[None], w)
        assert not g[2].any() and not g[3].any() and not g[4].any()


def test_shapes_streams_and_refusals():
    X = torch.randn(2, 33, 256, device=DEV).bfloat16()
    w = torch.ones(256, device=DEV).bfloat16()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    x, h = lac.stage_norm(X, X, w, None, w, p=0.1, seed=1, stream=s)
    y = lac.stage_dropout(X, 0.1, 1, stream=s)
    g = lac.stage_norm_bwd(X, X, x, X, w, None, w, p=0.1, seed=1, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    x2, h2 = lac.stage_norm(X.view(66, 256), X.view(66, 256), w, None, w, p=0.1, seed=1)
    assert torch.equal(x.view(66, 256), x2) and torch.equal(h.view(66, 256), h2)
    assert torch.equal(y, lac.stage_dropout(X, 0.1, 1))
    for a, b in zip(g, lac.stage_norm_bwd(X, X, x, X, w, None, w, p=0.1, seed=1)):
        assert a is b is None or torch.equal(a, b)
    for bad, status in ((dict(Y=X[:, :8]), -2), (dict(Y=X.float()), -3), (dict(Y=X, w_post=w[:8].contiguous()), -2),
                        (dict(Y=X.transpose(0, 1)), -2), (dict(Y=X, gate=torch.ones(5, 256, device=DEV).bfloat16()), -2),
                        (dict(p=0.5), -4), (dict(w_pre=w.cpu()), -1), (dict(store_x=False), -1)):
        with pytest.raises(lac.MaplError) as e:
            lac.stage_norm(X, **bad)
        assert e.value.status == status, bad


def test_edge_in_a_graph():
    a, kw, (gx, gh, x), first = check_edge(512, 1024, "bf16", True, True, 4, 0.1)
    ws = torch.empty(lac.stage_norm_bwd_workspace_bytes(512, 1024, 4), dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        xo, ho = lac.stage_norm(**a, **kw)
        out = lac.stage_norm_bwd(gx, gh, xo, a["Y"], a["w_post"], a["gate"], a["w_pre"], **kw, ws=ws)
        dr = lac.stage_dropout(gx, 0.1, 9)
    for turn in range(3):
        a["X"].copy_(torch.randn_like(a["X"]))
        ex, eh = lac.stage_norm(**a, **kw)
        want = lac.stage_norm_bwd(gx, gh, ex, a["Y"], a["w_post"], a["gate"], a["w_pre"], **kw)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(xo, ex) and torch.equal(ho, eh) and torch.equal(dr, lac.stage_dropout(gx, 0.1, 9))
        for s, t in zip(out, want):
            assert torch.equal(s, t)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_everything_dropped(dt):
    a, rng = edge_inputs(19, 333, dt, True, True, 1)
    a["Y"].fill_(float("nan"))
    x, h = lac.stage_norm(**a, p=1.0, seed=4)
    near(x, n64(a["X"]), np.abs(n64(a["X"])), DT[dt], 4, "X_out")
    assert h.isfinite().all()
    gx = rows(rng, 19, 333, dt)
    g = lac.stage_norm_bwd(gx, None, None, a["Y"], a["w_post"], a["gate"], None, p=1.0, seed=4)
    assert torch.equal(g[0], gx) and not g[1].any() and not g[2].any() and not g[3].any()


def test_empty_rows_with_the_smallest_eps():
    X = torch.zeros(5, 300, device=DEV)
    X[3] = 1e-20
    w = torch.ones(300, device=DEV)
    eps = float(torch.finfo(torch.float32).tiny)
    x, h = lac.stage_norm(X, X, w, None, w, eps=eps)
    g = lac.stage_norm_bwd(X + 1, X, x, X, w, None, w, eps=eps)
    assert x.isfinite().all() and h.isfinite().all() and not h[[0, 1, 2, 4]].any()
    assert all(t.isfinite().all() for t in (g[0], g[2], g[4]))
