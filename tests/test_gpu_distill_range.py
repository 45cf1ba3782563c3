"""The distillation loss at the edges of its inputs' range: logits far from zero,
where the loss is a difference of large numbers, teachers' logits of the lowest value,
and rows in several slices of which some hold nothing."""
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


def make(N, V, K, seed, step, size):
    """Logits that are multiples of `step` up to `size`, with labels and a teacher's entries of the same kind."""
    g = torch.Generator().manual_seed(seed)
    grid = lambda *s: torch.randint(-int(size / step), int(size / step) + 1, s, generator=g) * step  # noqa: E731
    Z, t = grid(N, V), grid(N, K)
    y, ids = (torch.randint(0, V, s, generator=g, dtype=torch.int32) for s in ((N,), (N, K)))
    return Z, y.to(DEV), ids.to(DEV), t


def sizes(z, t, T):
    """Sizes that the errors of a loss go by: of a cross-entropy's terms and of a divergence's."""
    span = np.max(z) - np.min(z)
    tspan = np.max(t) - np.min(t)
    return span, (span + tspan) / T


@pytest.mark.parametrize("N, V, K, T", [(5, 300, 9, 1.0), (5, 300, 9, 2.0), (3, 70001, 33, 1.5), (1100, 40, 3, 2.0)])
@pytest.mark.parametrize("offset", [2.0 ** 12, -2.0 ** 16])
def test_a_common_offset_does_not_count(N, V, K, T, offset):
    # multiples of 2^-6, exact in fp32 beside the offset; bf16 has no such numbers
    Z, y, ids, t = make(N, V, K, V, 2.0 ** -6, 8.0)
    want = block.distill(np64(Z), np64(y).astype(int), np64(ids).astype(int), np64(t), T, 0.5, 0.5)[0]
    ce, kd = sizes(np64(Z), np64(t), T)
    # a logarithm of a sum over V terms, by chains of at most V / 256 + 64 additions, and
    # differences of a few roundings each
    tol = ((V / 256 + 64) + 8 * ce + 8 * (kd + np.log(V))) * F32
    for z_off, t_off in ((offset, 0.0), (0.0, offset), (offset, -offset)):
        z, tt = (Z + z_off).to(DEV, torch.float32), (t + t_off).to(DEV, torch.float32)
        assert np.array_equal(np64(z) - z_off, np64(Z)) and np.array_equal(np64(tt) - t_off, np64(t))
        loss, stats = lac.stage_distill(z, y, ids, tt, T, 0.5, 0.5)
        off = np.abs(np64(loss) - want).max()
        assert off <= tol, (z_off, t_off, off, tol)


@pytest.mark.parametrize("N, V", [(4, 250), (3, 70000)])
def test_large_bf16_logits(N, V):
    # multiples of 2^8 from 2^15, where bf16 has them; a temperature that brings them together
    g = torch.Generator().manual_seed(V)
    Z = (2.0 ** 15 + 256 * torch.randint(0, 16, (N, V), generator=g)).to(DEV, torch.bfloat16)
    y, ids = (torch.randint(0, V, s, generator=g, dtype=torch.int32).to(DEV) for s in ((N,), (N, 8)))
    t, T = torch.randn(N, 8, generator=g) * 64, 64.0
    want = block.distill(np64(Z), np64(y).astype(int), np64(ids).astype(int), np64(t), T, 0.25, 1.0)[0]
    loss, _ = lac.stage_distill(Z, y, ids, t.to(DEV), T, 0.25, 1.0)
    # a cross-entropy of up to 3840 that is exact but for its rounding, and a divergence as above
    tol = 0.25 * 3840 * 2 * F32 + ((V / 256 + 64) + 8 * (60 + 6 + np.log(V))) * F32
    assert np.abs(np64(loss) - want).max() <= tol, np.abs(np64(loss) - want).max()


@pytest.mark.parametrize("T", [0.5, 1.0, 2.0])
@pytest.mark.parametrize("V", [100, 70000])
def test_teachers_entries_of_the_lowest_value(V, T):
    # the lowest value is a value: alone it is the row's teacher, beside others it weighs nothing
    Z, y, ids, t = make(3, V, 4, 3, 2.0 ** -6, 8.0)
    ids = torch.tensor([[1, 5, 9, 13]] * 3, dtype=torch.int32, device=DEV)
    Z, t, low = Z.to(DEV, torch.float32), t.to(DEV, torch.float32), torch.finfo(torch.float32).min
    t[0], t[1, 2:] = low, low
    even, two = t.clone(), ids.clone()
    even[0], two[1, 2:] = 0.0, -1
    a = lac.stage_distill(Z, y, ids, t, T)
    b = lac.stage_distill(Z, y, two, even, T)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    g = torch.ones(3, device=DEV)
    ga, gb = lac.stage_distill_bwd(g, Z, a[1], y, ids, t, T), lac.stage_distill_bwd(g, Z, b[1], y, two, even, T)
    assert torch.equal(ga, gb)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V", [70000, 131071])
@pytest.mark.parametrize("T", [1.0, 2.0])
def test_slices_that_hold_nothing(T, V, dt):
    # forward two and three slices a row, backward 17 and 31: some of them -inf throughout
    g = torch.Generator().manual_seed(V)
    N, K = 6, 5
    assert lac.stage_distill_workspace_bytes(N, V) > 0
    Z = (3 * torch.randn(N, V, generator=g)).clamp(-12, 12).to(DEV, DT[dt])
    Z[0, :V // 2] = -float("inf")             # the first slices
    Z[1, :-1], Z[1, -1] = -float("inf"), 2.0  # a single finite logit, the last
    Z[2, 3:] = torch.finfo(DT[dt]).min        # the lowest value from the third on
    Z[3, 8:] = -float("inf")                  # all but the first vector
    Z[4, V - 9:] = -float("inf")
    ids = torch.randint(0, V, (N, K), generator=g, dtype=torch.int32)
    y = torch.randint(0, V, (N,), generator=g, dtype=torch.int32)
    ids[0] = torch.arange(V - K, V)
    ids[1], y[1] = torch.tensor([V - 1, -1, V - 1, -1, -1]), V - 1
    ids[2], y[2] = torch.tensor([0, 1, 2, 1, -1]), 2
    ids[3], y[3] = torch.tensor([0, 7, 3, 4, 5]), 7
    ids[4], y[4], y[0] = torch.arange(K), V // 2, V - 2
    t, go = torch.randn(N, K, generator=g), torch.randn(N, generator=g)
    y, ids, t, go = (x.to(DEV) for x in (y, ids, t, go))
    a = (np64(y).astype(int), np64(ids).astype(int), np64(t), T, 0.5, 0.5)
    want, wstats, _ = block.distill(np64(Z), *a)
    loss, stats = lac.stage_distill(Z, y, ids, t, T, 0.5, 0.5)
    # finite logits of 12 in size: sums by chains of V / 256 + 64 additions, exponents and
    # differences of a few roundings each
    rel = (V / 256 + 64 + 8 * 24 * max(1.0, 1 / T) + 8 * np.log(V)) * F32
    assert np.all(np.abs(np64(stats) - wstats) <= 2 * rel)
    assert np.all(np.abs(np64(loss) - want) <= 4 * rel * (1 + np.abs(want)))
    gw, gsize = block.distill_bwd(np64(go), np64(Z), *a)
    gZ = lac.stage_distill_bwd(go, Z, stats, y, ids, t, T, 0.5, 0.5)
    half = 2.0 ** -8 if dt == "bf16" else F32
    assert np.all(np.abs(np64(gZ) - gw) <= 4 * rel * gsize + half * np.abs(gw) + 2.0 ** -126)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_slices_of_rows_do_not_mix(bad):
    # a value that is not finite in one slice reaches its own row, and no other
    g = torch.Generator().manual_seed(1)
    N, V = 4, 70000
    Z = torch.randn(N, V, generator=g).to(DEV)
    y = torch.randint(0, V, (N,), generator=g, dtype=torch.int32).to(DEV)
    go = torch.randn(N, generator=g).to(DEV)
    a = lac.stage_distill(Z, y)
    ga = lac.stage_distill_bwd(go, Z, a[1], y)
    Z[2, 60000] = bad
    b = lac.stage_distill(Z, y)
    gb = lac.stage_distill_bwd(go, Z, b[1], y)
    keep = [0, 1, 3]
    assert torch.equal(a[0][keep], b[0][keep]) and torch.equal(a[1][keep], b[1][keep]) and torch.equal(ga[keep], gb[keep])
    assert not torch.isfinite(b[0][2]) and not torch.isfinite(b[1][2]).any()
