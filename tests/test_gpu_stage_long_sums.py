"""Weight gradients of the block edge over many rows.

A thread adds up at most RUN rows in fp32 before its partial sum is joined with
the others in fp64, whatever the number of rows, so RUN additions count, each
off by at most half a step (2^-24) of a partial sum, which is at most the sum of
absolute values.  The factors of a term (reciprocal root, products) are STEPS
half steps more, and the result is rounded once."""
import pytest
import torch

import learned_activation_compression_amd as lac

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = torch.finfo(torch.float32).eps / 2
RUN, STEPS = 512, 16


def within(got, want, size, steps, what):
    bound = (steps + 1) * HALF * size
    err = (got.double() - want).abs()
    assert (err <= bound).all(), f"{what}: error {(err / size).max().item():.3e} of the sum's size, bound {steps * HALF:.3e}"


# one gate row, a few, many of long runs of rows, and more than a grid has rows of blocks
@pytest.mark.parametrize("N, G, d", [(1_000_003, 1, 1032), (2_600_000, 5, 1032), (1_200_000, 600, 136),
                                     (17_160_000, 33_000, 8)])
def test_small_terms_behind_a_large_one(N, G, d):
    # Rows of ones, whose norms are one; a gradient of 1.5 in the first row and of just under half a step of it in all
    # others: a sum that keeps running in fp32 loses every one of them.
    t = 251 / 256 * 2.0 ** -24
    g = torch.full((N, d), t, dtype=torch.bfloat16, device=DEV)
    g[0] = 1.5
    one = torch.ones(N, d, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(d, dtype=torch.bfloat16, device=DEV)
    gate = torch.ones(G, d, dtype=torch.bfloat16, device=DEV)
    unit = (1 + 1e-5) ** -0.5
    first = unit * (1.5 + (N // G - 1) * t)
    want = unit * (1.5 + (N - 1) * t)
    if G == 1:
        _, _, _, _, g_w_pre = lac.stage_norm_bwd(gH=g, X_out=one, w_pre=w, gX=torch.empty_like(g))
        within(g_w_pre, want, want, RUN + STEPS, "g_w_pre")
    _, _, g_w_post, g_gate, _ = lac.stage_norm_bwd(g, Y=one, w_post=w, gate=gate)
    within(g_w_post, want, want, RUN + STEPS, "g_w_post")
    within(g_gate[0], first, first, RUN + STEPS, "g_gate")
    if G > 1:
        rest = unit * (N // G) * t
        within(g_gate[1:], rest, rest, RUN + STEPS, "g_gate of the other rows")


@pytest.mark.parametrize("N, d, G, drop", [(300_003, 8192, 0, 0.0), (300_000, 2048, 4, 0.1), (270_000, 1000, 900, 0.1),
                                           (1_100_000, 72, 550, 0.0), (530_000, 520, 530_000, 0.0)])
def test_weight_gradients_against_sums_in_fp64(N, d, G, drop):
    gen = torch.Generator(device=DEV).manual_seed(N + d)

    def randn(*s):
        return torch.randn(*s, dtype=torch.bfloat16, device=DEV, generator=gen)

    Y, x, h, gx = randn(N, d), randn(N, d), randn(N, d), randn(N, d)
    wp, wq = 1 + 0.2 * randn(d), 1 + 0.2 * randn(d)
    gate = 1 + 0.2 * randn(G, d) if G else None
    if drop:  # the mask, from ones
        keep = lac.stage_dropout(torch.ones_like(Y), drop, 9, 5)
    _, gY, g_w_post, g_gate, g_w_pre = lac.stage_norm_bwd(gx, h, x, Y, wp, gate, wq, gX=torch.empty_like(x), p=drop, seed=9,
                                                          offset=5)
    del gY
    ref = {k: torch.zeros(s, dtype=torch.float64, device=DEV) for k, s in
           (("w_post", d), ("w_pre", d), ("gate", (max(G, 1), d)))}
    size = {k: torch.zeros_like(v) for k, v in ref.items()}
    scale = 65536 / (65536 - int(drop * 65536 + 0.5))
    per = N // max(G, 1)
    chunk = 1 << 27 >> (d - 1).bit_length()
    for r0 in range(0, N, chunk):
        s = slice(r0, min(r0 + chunk, N))
        X, H, T, u = (v[s].double() for v in (x, h, gx, Y))
        r = (X.square().mean(1, keepdim=True) + 1e-5).rsqrt()
        a = H * wq.double()
        t = T + r * (a - X * r * r * (a * X).mean(1, keepdim=True))
        # the size of the terms of t: an error of its parts counts against them
        big = T.abs() + r * (a.abs() + X.abs() * r * r * (a * X).abs().mean(1, keepdim=True))
        if drop:
            u = u * (keep[s] != 0) * scale
        u = u * (u.square().mean(1, keepdim=True) + 1e-5).rsqrt()
        row = torch.arange(s.start, s.stop, device=DEV) // per
        g = gate[row].double() if G else 1.0
        ref["w_pre"] += (H * X * r).sum(0)
        size["w_pre"] += (H * X * r).abs().sum(0)
        ref["w_post"] += (t * g * u).sum(0)
        size["w_post"] += (big * g * u).abs().sum(0)
        lo, hi = s.start // per, (s.stop - 1) // per
        for k in range(lo, hi + 1) if G and hi - lo < 64 else ():
            m = slice(max(k * per, s.start) - s.start, min((k + 1) * per, s.stop) - s.start)
            ref["gate"][k] += (t[m] * wp.double() * u[m]).sum(0)
            size["gate"][k] += (big[m] * wp.double() * u[m]).abs().sum(0)
        if G and hi - lo >= 64:
            ref["gate"].index_add_(0, row, t * wp.double() * u)
            size["gate"].index_add_(0, row, (big * wp.double() * u).abs())
    steps = RUN + 4 * (d / 8 + 32)  # and the sums of the row, each by its size
    within(g_w_pre, ref["w_pre"], size["w_pre"], steps, "g_w_pre")
    within(g_w_post, ref["w_post"], size["w_post"], steps, "g_w_post")
    if G:
        within(g_gate, ref["gate"], size["gate"], steps, "g_gate")
