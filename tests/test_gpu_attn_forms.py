"""Causal attention in each of the forms that the number of rows and heads
selects (blocks of 128 rows, blocks of 32 whose waves share the keys, a backward
range that is split and joined), against float64 products on the device."""
import numpy as np
import pytest
import torch

import learned_activation_compression_amd as lac

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
F32 = 2.0 ** -24


def make(lens, Hq, Hkv, D, dt, seed, pad=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    N = sum(lens)
    x = torch.randn(N, (2 * Hq + 2 * Hkv) * D + pad, generator=g, device=DEV)
    x[:, :(Hq + Hkv) * D] *= 1.4
    x = x.to(DT[dt])
    a, b, c = Hq * D, (Hq + Hkv) * D, (Hq + 2 * Hkv) * D
    cu = torch.tensor(np.cumsum([0, *lens]), dtype=torch.int32, device=DEV)
    return (x[:, :a].unflatten(1, (Hq, D)), x[:, a:b].unflatten(1, (Hkv, D)), x[:, b:c].unflatten(1, (Hkv, D)),
            x[:, c:c + a].unflatten(1, (Hq, D)), cu)


def reference(q, k, v, go, lens, scale):
    """o, lse, gradients and the sizes that errors go by, head by head in float64."""
    N, Hq, D = q.shape
    G = Hq // k.shape[1]
    f = lambda x: x.double()  # noqa: E731
    out = {n: torch.zeros(s, dtype=torch.float64, device=DEV) for n, s in
           (("o", q.shape), ("gq", q.shape), ("gk", k.shape), ("gv", v.shape), ("lse", (Hq, N)))}
    size = {n: torch.zeros_like(x) for n, x in out.items()}
    at = 0
    for n in lens:
        if n == 0:
            continue
        r = slice(at, at + n)
        seen = torch.ones(n, n, dtype=torch.bool, device=DEV).tril()
        for h in range(Hq):
            Q, K, V, g = f(q[r, h]).contiguous(), f(k[r, h // G]).contiguous(), f(v[r, h // G]).contiguous(), f(go[r, h])
            s = (scale * (Q @ K.t().contiguous())).masked_fill(~seen, -torch.inf)
            lse = torch.logsumexp(s, 1, keepdim=True)
            p = torch.exp(s - lse)
            o = p @ V
            dp = g @ V.t().contiguous()
            dd = (g * o).sum(1, keepdim=True)
            ds = scale * p * (dp - dd)
            dz = scale * p * (g.abs() @ V.abs().t().contiguous() + (g * o).abs().sum(1, keepdim=True))
            out["o"][r, h], out["lse"][h, r] = o, lse[:, 0]
            size["o"][r, h] = p @ V.abs()
            size["lse"][h, r] = (scale * (Q.abs() @ K.abs().t().contiguous())).masked_fill(~seen, 0).amax(1)
            out["gq"][r, h], size["gq"][r, h] = ds @ K, dz @ K.abs()
            out["gk"][r, h // G] += ds.t().contiguous() @ Q
            out["gv"][r, h // G] += p.t().contiguous() @ g
            size["gk"][r, h // G] += dz.t().contiguous() @ Q.abs()
            size["gv"][r, h // G] += p.t().contiguous() @ g.abs()
        at += n
    return out, size


def check(got, want, size, rel, dt, name):
    # rel: the fp32 errors of scores, weights and sums, relative to the sum of sizes; bf16:
    # a factor's rounding, half a step of that sum, and the output's
    half = 2.0 ** -8 if dt == "bf16" else 0.0
    tol = size * (rel + half) + want.abs() * (half + F32) + 1e-30
    off = (got.double() - want).abs()
    assert torch.isfinite(got).all() and torch.all(off <= tol), (name, (off - tol).max().item())


def run(lens, Hq, Hkv, D, dt, seed=1, pad=0):
    q, k, v, go, cu = make(lens, Hq, Hkv, D, dt, seed, pad)
    scale = D ** -0.5
    O, lse = lac.stage_attn(q, k, v, cu)
    g = lac.stage_attn_bwd(go, q, k, v, O, lse, cu)
    want, size = reference(q, k, v, go, lens, scale)
    worst, n = size["lse"].max().item(), max(lens)
    rel = (2 * (D + 4) * worst + n + 8) * F32
    check(O, want["o"], size["o"], rel, dt, "o")
    off = (lse.double() - want["lse"]).abs()
    assert torch.all(off <= ((D + 4) * 1.01 * size["lse"] + 4 * want["lse"].abs() + n + 8) * F32)
    # delta is taken from the stored O: its rounding enters each term
    rel = (2 * (D + 4) * worst + 4 * lse.abs().max().item() + 2 * D + n * (Hq // Hkv) + 16) * F32
    rel += 2.0 ** -8 if dt == "bf16" else F32
    for x, name in zip(g, ("gq", "gk", "gv")):
        check(x, want[name], size[name], rel, dt, name)
    return q, k, v, go, cu, O, lse, g


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("lens, Hq, Hkv, D", [
    ([2100], 16, 4, 64),                       # 272 blocks of 128 rows; the backward split over keys and heads
    ([700, 1, 900, 0, 63, 65, 400], 16, 16, 80),
    ([1025, 1024], 24, 8, 128),
    ([513] * 9, 8, 8, 64),
    ([64] * 70, 8, 4, 96),                     # two sequences in each block
    ([7] * 600, 8, 2, 32),                     # many in each
])
def test_blocks_of_128_rows(lens, Hq, Hkv, D, dt):
    run(lens, Hq, Hkv, D, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("lens, Hq, Hkv, D", [([1999], 2, 1, 64), ([1500, 3, 700], 4, 1, 128), ([130] * 12, 3, 1, 80),
                                              ([33, 1, 31, 32], 1, 1, 64)])
def test_few_rows_and_split_ranges(lens, Hq, Hkv, D, dt):
    run(lens, Hq, Hkv, D, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D, pad", [(63, 1), (64, 3), (100, 1), (127, 0)])
def test_rows_at_any_address_in_large_blocks(D, pad, dt):
    run([1000, 1200], 16, 2, D, dt, pad=pad)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("lens, Hq, Hkv", [([900, 900, 400], 16, 8), ([200, 100], 2, 1)])
def test_unseen_values_in_every_form(lens, Hq, Hkv, dt):
    q, k, v, go, cu, O, lse, g = run(lens, Hq, Hkv, 64, dt)
    N, a, b = sum(lens), lens[0] + 37, lens[0] + 40
    k, v, go = k.clone(), v.clone(), go.clone()
    k[a:b], v[a + 1:b], go[a - 20] = float("nan"), float("inf"), float("nan")
    O2, lse2 = lac.stage_attn(q, k, v, cu)
    n = torch.arange(N, device=DEV)
    end = lens[0] + lens[1]
    spoilt = (n >= a) & (n < end)  # the rows that see row a
    assert torch.isnan(O2[spoilt]).all() and torch.isfinite(O2[~spoilt]).all() and torch.isfinite(lse2[:, ~spoilt]).all()
    # a row computed again adds up in another order; bf16 weights are not rounded then
    tol = 2.0 ** -6 if dt == "bf16" else 1e-5
    assert torch.all((O2 - O)[~spoilt].abs().float() <= tol * (1 + O[~spoilt].abs().float()))
    g2 = lac.stage_attn_bwd(go, q, k, v, O2, lse2, cu)
    bad_q = spoilt | (n == a - 20)
    bad_k = (n >= lens[0]) & (n < end)
    for x, y, bad in zip(g2, g, (bad_q, bad_k, bad_k)):
        assert torch.isnan(x[bad]).all() and torch.isfinite(x[~bad]).all()
        top = y.float().abs().max()
        assert torch.all((x - y)[~bad].abs().float() <= (2.0 ** -6 if dt == "bf16" else 1e-5) * top)


def test_repeats_bit_for_bit():
    for lens, Hq, Hkv in (([2100], 16, 4), ([300, 50], 2, 1)):
        q, k, v, go, cu = make(lens, Hq, Hkv, 64, "bf16", 3)
        a = lac.stage_attn(q, k, v, cu)
        a += lac.stage_attn_bwd(go, q, k, v, *a, cu)
        for _ in range(3):
            b = lac.stage_attn(q, k, v, cu)
            b += lac.stage_attn_bwd(go, q, k, v, *b, cu)
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_gradient_against_differences():
    # fp32, along random directions: central differences of the loss in float64 sums
    lens, Hq, Hkv, D = [40, 90], 4, 2, 64
    q, k, v, go, cu = make(lens, Hq, Hkv, D, "f32", 5)
    q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    O, lse = lac.stage_attn(q, k, v, cu)
    grads = lac.stage_attn_bwd(go.contiguous(), q, k, v, O, lse, cu)
    loss = lambda *x: (lac.stage_attn(*x, cu)[0].double() * go.double()).sum().item()  # noqa: E731
    gen = torch.Generator(device=DEV).manual_seed(6)
    for i, (x, gx) in enumerate(zip((q, k, v), grads)):
        d = torch.randn(x.shape, generator=gen, device=DEV)
        step = 2.0 ** -7
        args = [q, k, v]
        args[i] = x + step * d
        hi = loss(*args)
        args[i] = x - step * d
        lo = loss(*args)
        num, got = (hi - lo) / (2 * step), (gx.double() * d.double()).sum().item()
        # the loss's fp32 errors over the step, and step^2 times third derivatives
        size = (O.double() * go.double()).abs().sum().item()
        assert abs(num - got) <= 64 * F32 * size / step + 30 * step ** 2 * size / lens[1] ** 0.5, (i, num, got)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N", [2049, 2080, 2081, 2112, 2145, 2175])
def test_last_block_of_every_fill(N, dt):
    # the last block of 128 rows holds 1 to 127 of them: some of its waves have no row
    run([N - 20, 20], 16, 4, 64, dt, seed=N)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [2.0 ** -64, 2.0 ** -20, 40.0])
def test_scales_at_their_ends(scale, dt):
    lens, Hq, Hkv, D = [300, 40], 2, 1, 64
    q, k, v, go, cu = make(lens, Hq, Hkv, D, dt, 7)
    O, lse = lac.stage_attn(q, k, v, cu, scale)
    g = lac.stage_attn_bwd(go, q, k, v, O, lse, cu, scale)
    want, size = reference(q, k, v, go, lens, scale)
    rel = (2 * (D + 4) * size["lse"].max().item() + max(lens) + 8) * F32
    check(O, want["o"], size["o"], min(rel, 1.0), dt, "o")
    rel = (2 * (D + 4) * size["lse"].max().item() + 4 * lse.abs().max().item() + 2 * D + 2 * max(lens) + 16) * F32
    rel += 2.0 ** -8 if dt == "bf16" else F32
    for x, name in zip(g, ("gq", "gk", "gv")):
        check(x, want[name], size[name], min(rel, 2.0), dt, name)


def test_two_calls_at_once():
    # two streams, a workspace each: what one leaves in its own does not reach the other
    lens, Hq, Hkv, D = [1999], 2, 1, 64
    a, b = make(lens, Hq, Hkv, D, "bf16", 1), make([700, 1299], Hq, Hkv, D, "bf16", 2)

    def both(x, stream=None):
        q, k, v, go, cu = x
        O, lse = lac.stage_attn(q, k, v, cu, stream=stream)
        return (O, lse, *lac.stage_attn_bwd(go, q, k, v, O, lse, cu, stream=stream))

    want = [both(a), both(b)]
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    got = [[], []]
    for _ in range(4):
        got[0].append(both(a, s))
        got[1].append(both(b, t))
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        for r in runs:
            assert all(torch.equal(x, y) for x, y in zip(w, r))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("Hq, Hkv, D, pad", [(4, 2, 128, 0), (6, 2, 40, 1), (256, 256, 16, 0)])
def test_unseen_values_beside_many_that_are_seen(Hq, Hkv, D, pad, dt):
    # a row whose sum an unseen NaN has spoilt is formed again over hundreds of visible rows
    lens = [300, 190]
    q, k, v, go, cu, O, lse, _ = run(lens, Hq, Hkv, D, dt, pad=pad)
    want, size = reference(q, k, v, go, lens, D ** -0.5)
    worst, n = size["lse"].max().item(), max(lens)
    rel = (2 * (D + 4) * worst + n + 8) * F32
    others = lambda i: torch.arange(sum(lens), device=DEV) != i  # noqa: E731
    last, first = others(299), others(300)
    v2 = v.clone()
    v2[299] = float("inf")  # seen by row 299 alone
    O2, lse2 = lac.stage_attn(q, k, v2, cu)
    check(O2[last], want["o"][last], size["o"][last], rel, dt, "o")
    assert not torch.isfinite(O2[299]).any() and torch.all((lse2 - lse).abs() <= rel * (1 + lse.abs()))
    rel = (2 * (D + 4) * worst + 4 * lse.abs().max().item() + 2 * D + n * (Hq // Hkv) + 16) * F32
    rel += 2.0 ** -8 if dt == "bf16" else F32
    gq, gk, gv = lac.stage_attn_bwd(go, q, k, v2, O, lse, cu)
    check(gq[last], want["gq"][last], size["gq"][last], rel, dt, "gq")
    check(gk[last], want["gk"][last], size["gk"][last], rel, dt, "gk")
    check(gv, want["gv"], size["gv"], rel, dt, "gv")
    assert not torch.isfinite(gk[299]).any() and not torch.isfinite(gq[299]).any()  # the only pair of key 299
    go2 = go.clone()
    go2[300] = float("nan")  # a factor of key 300's gradients alone
    gq, gk, gv = lac.stage_attn_bwd(go2, q, k, v, O, lse, cu)
    check(gq[first], want["gq"][first], size["gq"][first], rel, dt, "gq")
    check(gk[first], want["gk"][first], size["gk"][first], rel, dt, "gk")
    check(gv[first], want["gv"][first], size["gv"][first], rel, dt, "gv")
    assert torch.isnan(gq[300]).all() and torch.isnan(gk[300]).all() and torch.isnan(gv[300]).all()
