"""Causal attention over packed sequences and its backward pass against the
float64 oracle: types, head layouts, widths, lengths, strides, rows of no
sequence, values that are not finite in places that a row does not see."""
import numpy as np
import pytest
import torch

import learned_activation_compression_amd as lac
from oracle import block

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
F32 = 2.0 ** -24  # half a step, relative


def np64(t):
    return t.detach().cpu().double().numpy()


def edges(lens, first=0):
    return torch.tensor(np.cumsum([first, *lens]), dtype=torch.int32, device=DEV)


def make(N, Hq, Hkv, D, dt, seed=0, pad=0, spread=1.5):
    """q, k, v, go as columns of one fused tensor with `pad` more columns, and cast to dt."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(N, (2 * Hq + 2 * Hkv) * D + pad, generator=g)
    x[:, :(Hq + Hkv) * D] *= spread
    x = x.to(DEV, DT[dt])
    a, b, c = Hq * D, (Hq + Hkv) * D, (Hq + 2 * Hkv) * D
    return (x[:, :a].unflatten(1, (Hq, D)), x[:, a:b].unflatten(1, (Hkv, D)), x[:, b:c].unflatten(1, (Hkv, D)),
            x[:, c:c + a].unflatten(1, (Hq, D)))


TINY = 2.0 ** -126  # what is smaller may count as zero


def fwd_bound(dt, o, size, ssize, n, D, vtop):
    """What each output may be off.  fp32: a score is off by (D + 4) half steps of the
    sum of its products' sizes (the products' sum, the scale, the exponent's two
    roundings), a weight relatively by twice that (itself and the row's sum), and the
    sums over n keys by n + 8 half steps.  A weight or a product below the smallest normal
    number may be dropped: n times that, times the largest factor.  bf16: the weights'
    rounding, half a step of the sum of sizes, and the output's."""
    rel = 2 * (D + 4) * F32 * ssize.T[..., None] * 1.01 + (n + 8) * F32
    tol = size * rel + np.abs(o) * F32 + n * TINY * (1 + vtop)
    if dt == "bf16":
        tol = tol + size * 2.0 ** -8 + np.abs(o) * 2.0 ** -8
    return tol


def bwd_bound(dt, g, size, ssize, lse, n, D, top):
    """As fwd_bound; a weight's error also has the rounding of the log-sum (to fp32, times
    log2 e, and in the exponent), and a term's difference the errors of two sums over D.
    `top` is the largest factor that a dropped weight could have had, a product of three
    inputs summed over D.  bf16: the factor's rounding, half a step, and the gradient's."""
    worst = np.nanmax(ssize)
    rel = (2 * (D + 4) * worst + 4 * np.nanmax(np.abs(lse)) + 2 * D + n + 16) * F32
    tol = size * rel + np.abs(g) * F32 + n * TINY * (1 + top)
    if dt == "bf16":
        tol = tol + size * 2.0 ** -8 + np.abs(g) * 2.0 ** -8
    return tol


def check(name, got, want, tol):
    got = np64(got)
    ok = np.isfinite(want)
    assert np.array_equal(np.isfinite(got)[ok], ok[ok]), name
    off = np.abs(got - want)[ok] - tol[ok]
    assert off.size == 0 or off.max() <= 0, (name, off.max(), np.abs(got - want)[ok].max())


def run_both(q, k, v, go, cu, dt, scale=None, lens=None, **kw):
    N, Hq, D = q.shape
    c = D ** -0.5 if scale is None else scale
    O, lse = lac.stage_attn(q, k, v, cu, scale)
    qn, kn, vn, gn, cn = np64(q), np64(k), np64(v), np64(go), cu.cpu().numpy()
    o, l, size, ssize = block.attn(qn, kn, vn, cn, c)
    n = int(np.max(np.diff(cn), initial=1))
    inside = block.starts(cn, N) >= 0
    check("O", O[torch.from_numpy(inside)], o[inside], fwd_bound(dt, o, size, ssize, n, D, np.nanmax(np.abs(vn)))[inside])
    ltol = ((D + 4) * 1.01 * ssize + 4 * np.abs(l) + n + 8) * F32
    check("lse", lse[:, torch.from_numpy(inside)], l[:, inside], ltol[:, inside])
    gs = lac.stage_attn_bwd(go, q, k, v, O, lse, cu, scale)
    On, ln = np64(O), np64(lse)
    g, gsize = block.attn_bwd(gn, qn, kn, vn, On, ln, cn, c)
    a = [np.nanmax(np.abs(x[inside])) for x in (qn, kn, vn, gn, On)]
    top = max(1.0, 2 * D * max(a[2], a[4])) * a[3] * max(a[0], a[1], 1.0)
    for name, got in zip(("gq", "gk", "gv"), gs):
        sel = torch.from_numpy(inside)
        check(name, got[sel], g[name][inside],
              bwd_bound(dt, g[name], gsize[name], ssize, l, n * (Hq // k.shape[1]), D, top)[inside])
    return O, lse, gs


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("lens, Hq, Hkv, D", [
    ([1], 1, 1, 64), ([2], 2, 1, 32), ([33], 2, 2, 64), ([64], 4, 1, 128), ([129], 3, 3, 96), ([200], 8, 2, 80),
    ([1, 1, 1, 1, 1], 2, 1, 64), ([5, 0, 31, 1, 0, 64, 100], 6, 2, 64), ([127, 128, 1], 2, 2, 128),
    ([300], 4, 2, 72), ([31, 32, 33], 1, 1, 8), ([257, 63], 2, 1, 40), ([400, 13], 1, 1, 112),
])
def test_against_the_oracle(lens, Hq, Hkv, D, dt):
    q, k, v, go = make(sum(lens), Hq, Hkv, D, dt, seed=sum(lens) + D)
    run_both(q, k, v, go, edges(lens), dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D, pad", [(1, 0), (7, 0), (33, 1), (50, 0), (64, 1), (64, 3), (77, 2), (96, 1), (127, 0),
                                    (128, 2), (128, 5)])
def test_any_width_and_stride(D, pad, dt):
    # rows and heads that begin anywhere
    lens = [3, 90, 41]
    q, k, v, go = make(sum(lens), 4, 2, D, dt, seed=D + pad, pad=pad)
    run_both(q, k, v, go, edges(lens), dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_of_no_sequence_are_left(dt):
    lens, N = [40, 17, 70], 300
    q, k, v, go = make(N, 4, 2, 64, dt, seed=5)
    cu = edges(lens, first=35)
    inside = torch.from_numpy(block.starts(cu.cpu().numpy(), N) >= 0)
    O = torch.full((N, 4, 64), 7.0, dtype=DT[dt], device=DEV)
    lse = torch.full((4, N), 7.0, device=DEV)
    outs = [torch.full(x.shape, 7.0, dtype=DT[dt], device=DEV) for x in (q, k, v)]
    # what is there does not count, whatever it is
    for x in (q, k, v, go):
        x[~inside] = float("nan")
    lac.stage_attn(q, k, v, cu, O=O, lse=lse)
    assert torch.all(O[~inside] == 7) and torch.all(lse[:, ~inside] == 7)
    lac.stage_attn_bwd(go, q, k, v, O, lse, cu, gQ=outs[0], gK=outs[1], gV=outs[2])
    for x in outs:
        assert torch.all(x[~inside] == 7) and torch.isfinite(x).all()
    run_both(q, k, v, go, cu, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("what", ["k", "v", "kv"])
def test_unseen_values_do_not_count(dt, bad, what):
    # the second sequence and the end of the third are spoilt: no other row changes
    lens = [50, 20, 100]
    q, k, v, go = make(sum(lens), 4, 2, 64, dt, seed=9)
    cu = edges(lens)
    clean, clse = lac.stage_attn(q, k, v, cu)
    rows = [*range(55, 70), 169]
    for n, x in (("k", k), ("v", v)):
        if n in what:
            x[rows] = bad
    O, lse = lac.stage_attn(q, k, v, cu)
    keep = torch.ones(sum(lens), dtype=torch.bool)
    keep[55:70] = keep[169] = False
    tol = 2.0 ** -8 if dt == "bf16" else 1e-5  # a row computed again adds up in another order
    d = (O[keep].float() - clean[keep].float()).abs()
    assert torch.all(d <= 2 * tol * clean[keep].float().abs() + tol)
    torch.testing.assert_close(lse[:, keep], clse[:, keep], rtol=1e-5, atol=1e-5)
    want = block.attn(np64(q), np64(k), np64(v), cu.cpu().numpy(), 0.125)
    got = np64(O)
    assert np.array_equal(np.isnan(got), np.isnan(want[0])) and np.array_equal(np.isinf(got), np.isinf(want[0]))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_unseen_gradients_do_not_count(dt):
    # gO of one row in the middle is NaN: it reaches its own gQ and the keys that it sees
    lens = [50, 60, 40]
    q, k, v, go = make(sum(lens), 2, 1, 64, dt, seed=11)
    cu = edges(lens)
    O, lse = lac.stage_attn(q, k, v, cu)
    clean = lac.stage_attn_bwd(go, q, k, v, O, lse, cu)
    go[80] = float("nan")
    got = lac.stage_attn_bwd(go, q, k, v, O, lse, cu)
    n = torch.arange(sum(lens), device=DEV)
    spoilt = {"gq": n == 80, "gk": (n >= 50) & (n <= 80), "gv": (n >= 50) & (n <= 80)}
    for (name, bad), x, y in zip(spoilt.items(), got, clean):
        assert torch.isnan(x[bad]).all() and torch.isfinite(x[~bad]).all(), name
        d = (x[~bad].float() - y[~bad].float()).abs()
        # the sums' order and, in bf16, the factors' rounding
        top = y.float().abs().max()
        assert torch.all(d <= (2.0 ** -6 if dt == "bf16" else 1e-5) * top), name


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_scores_of_any_size(dt):
    # scores in the hundreds: one key has all the weight; and all of them alike
    lens = [70, 30]
    q, k, v, go = make(sum(lens), 2, 2, 64, dt, seed=3, spread=12.0)
    run_both(q, k, v, go, edges(lens), dt)
    q.zero_()
    run_both(q, k, v, go, edges(lens), dt)
    # a score of -inf has no weight beside others; alone it makes its row NaN, as the formula
    q.fill_(1.0)
    k.fill_(0.5)
    k[5] = -float("inf")
    O, lse = lac.stage_attn(q, k, v, edges(lens))
    o = block.attn(np64(q), np64(k), np64(v), np.array([0, 70, 100]), 0.125)[0]
    assert np.isfinite(o).all() and torch.isfinite(O).all()
    assert np.abs(np64(O) - o).max() <= 2.0 ** -6
    k[70] = -float("inf")
    O, lse = lac.stage_attn(q, k, v, edges(lens))
    assert torch.isnan(O[70]).all() and torch.isfinite(O[:70]).all() and torch.isfinite(O[71:]).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_scale_and_repeats(dt):
    lens = [90, 200, 7]
    q, k, v, go = make(sum(lens), 6, 2, 64, dt, seed=21)
    a = run_both(q, k, v, go, edges(lens), dt, scale=0.031)
    b = run_both(q, k, v, go, edges(lens), dt, scale=0.031)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert all(torch.equal(x, y) for x, y in zip(a[2], b[2]))


def test_more_edges_than_fit_on_chip():
    # 3000 sequences of one and two rows
    lens = [1 + i % 2 for i in range(3000)]
    q, k, v, go = make(sum(lens), 1, 1, 8, "f32", seed=2)
    run_both(q, k, v, go, edges(lens), "f32")


def test_edges_that_break_the_rules_stay_inside():
    N = 200
    q, k, v, go = make(N, 2, 1, 64, "bf16", seed=4)
    big = torch.full((3, N, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    for bad in ([0, 500], [-50, 100, 400], [150, 50, 180], [2 ** 31 - 1, 0], [-2 ** 31, 2 ** 31 - 1]):
        cu = torch.tensor(bad, dtype=torch.int32, device=DEV)
        O, lse = lac.stage_attn(q, k, v, cu, O=big[1])
        g = lac.stage_attn_bwd(go, q, k, v, O, lse, cu)
        torch.cuda.synchronize()
        assert torch.all(big[0] == 7) and torch.all(big[2] == 7) and len(g) == 3


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gradients_of_columns_of_one_tensor(dt):
    lens, Hq, Hkv, D = [65, 40], 4, 2, 64
    N = sum(lens)
    q, k, v, go = make(N, Hq, Hkv, D, dt, seed=8)
    O, lse = lac.stage_attn(q, k, v, edges(lens))
    plain = lac.stage_attn_bwd(go, q, k, v, O, lse, edges(lens))
    g = torch.full((N, (Hq + 2 * Hkv) * D + 8), 7.0, dtype=DT[dt], device=DEV)
    views = [x.unflatten(1, (-1, D)) for x in g[:, :-8].split([Hq * D, Hkv * D, Hkv * D], dim=1)]
    lac.stage_attn_bwd(go, q, k, v, O, lse, edges(lens), gQ=views[0], gK=views[1], gV=views[2])
    assert all(torch.equal(x, y) for x, y in zip(views, plain)) and torch.all(g[:, -8:] == 7)


def test_long_sequences_against_float64_rows():
    # 5000 keys: rows picked over the whole range
    N, Hq, Hkv, D = 5000, 2, 1, 128
    q, k, v, go = make(N, Hq, Hkv, D, "bf16", seed=13)
    cu = edges([N])
    O, lse = lac.stage_attn(q, k, v, cu)
    for i in (0, 1, 63, 64, 1000, 2047, 2048, 4095, 4999):
        s = (k[:i + 1, 0].double() @ q[i].double().t()) * D ** -0.5
        p = torch.softmax(s, 0)
        want, size = p.t() @ v[:i + 1, 0].double(), p.t() @ v[:i + 1, 0].double().abs()
        tol = 2.0 ** -8 * (want.abs() + size) + 2.0 ** -12 * size
        assert torch.all((O[i].double() - want).abs() <= tol), i
        torch.testing.assert_close(lse[:, i].double(), torch.logsumexp(s, 0), rtol=1e-5, atol=1e-5)


def test_streams_graphs_and_errors():
    lens = [100, 60]
    q, k, v, go = make(sum(lens), 2, 1, 64, "bf16", seed=17)
    cu = edges(lens)
    O, lse = lac.stage_attn(q, k, v, cu)
    g = lac.stage_attn_bwd(go, q, k, v, O, lse, cu)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    O2, lse2 = lac.stage_attn(q, k, v, cu, stream=s)
    g2 = lac.stage_attn_bwd(go, q, k, v, O2, lse2, cu, stream=s)
    s.synchronize()
    assert torch.equal(O, O2) and torch.equal(lse, lse2) and all(torch.equal(x, y) for x, y in zip(g, g2))
    out = [torch.zeros_like(x) for x in (O, lse, *g)]
    ws = torch.empty(lac.stage_attn_bwd_workspace_bytes(sum(lens), 2, 1, 64), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lac.stage_attn(q, k, v, cu, O=out[0], lse=out[1])
        lac.stage_attn_bwd(go, q, k, v, out[0], out[1], cu, gQ=out[2], gK=out[3], gV=out[4], ws=ws)
    for turn in range(3):
        for x in out:
            x.zero_()
        q.mul_(0.5)
        want = lac.stage_attn(q, k, v, cu)
        want += lac.stage_attn_bwd(go, q, k, v, *want, cu)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want)), turn
    for call in (lambda: lac.stage_attn(q, k, v.float(), cu), lambda: lac.stage_attn(q, k, v, cu.long()),
                 lambda: lac.stage_attn(q, k, v[:, :, :32], cu), lambda: lac.stage_attn(q, k, v, cu, scale=0.0),
                 lambda: lac.stage_attn(q.transpose(0, 1), k, v, cu), lambda: lac.stage_attn(q, k, v.cpu(), cu),
                 lambda: lac.stage_attn(q.half(), k.half(), v.half(), cu),
                 lambda: lac.stage_attn(torch.cat([q, q[:, :1]], 1), torch.cat([k, k], 1), torch.cat([v, v], 1), cu),
                 lambda: lac.stage_attn_bwd(go, q, k, v, O, lse[:, :-1], cu),
                 lambda: lac.stage_attn_bwd(go, q, k, v, O, lse, cu, ws=ws[:-1])):
        with pytest.raises(lac.MaplError):
            call()
