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
