"""The distillation loss and its gradient against the float64 oracle."""
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
    return None if t is None else t.detach().cpu().double().numpy()


def make(N, V, K, dt, seed=0, spread=3.0, t_spread=3.0):
    g = torch.Generator().manual_seed(seed)
    Z = (spread * torch.randn(N, V, generator=g)).to(DEV, DT[dt])
    ids = torch.randint(0, V, (N, K), generator=g, dtype=torch.int32)
    t = t_spread * torch.randn(N, K, generator=g)
    y = torch.randint(0, V, (N,), generator=g, dtype=torch.int32)
    y[torch.rand(N, generator=g) < 0.2] = -1
    ids[torch.rand(N, K, generator=g) < 0.1] = -1
    return Z, y.to(DEV), ids.to(DEV), t.to(DEV), torch.randn(N, generator=g).to(DEV)


def run_both(Z, y, ids, t, g, T=1.0, w_ce=1.0, w_kd=1.0):
    kw = dict(labels=y, t_ids=ids, t_logits=t, temperature=T, w_ce=w_ce, w_kd=w_kd)
    loss, stats = lac.stage_distill(Z, **kw)
    gZ = lac.stage_distill_bwd(g, Z, stats, **kw)
    N, V = Z.shape
    no = np.zeros((N, 0))
    a = (np64(y), no.astype(int) if ids is None else ids.cpu().numpy(), no if t is None else np64(t), T, w_ce, w_kd)
    a = (None if a[0] is None else a[0].astype(int), *a[1:])
    zn = np64(Z)
    want, wstats, size = block.distill(zn, *a)
    entries = no if t is None else np64(t)[np.isfinite(np64(t))]
    top = np.max(np.abs(zn), initial=1.0) * max(1.0, 1.0 / T) + np.max(np.abs(entries), initial=0) / T
    # an exponent is off by a few half steps of its size, a sum of n terms by what its
    # longest chain of additions rounds (at most n / 256 + 64), relatively
    rel = (8 * top + V / 256 + 64) * F32
    got = np64(stats)
    assert np.all(np.abs(got - wstats) <= rel + 2 * np.abs(wstats) * F32), np.abs(got - wstats).max()
    off = np.abs(np64(loss) - want)
    assert np.all(off <= (abs(w_ce) + abs(w_kd) * (1 + 4 * top)) * rel + 8 * size * F32), off.max()
    gw, gsize = block.distill_bwd(np64(g), zn, *a)
    # a softmax is off by its exponent's error and the log-sum's, an entry's weight by as much
    tol = gsize * (2 * rel + 8 * top * F32 + 8 * F32) + 2.0 ** -126
    tol += np.abs(gw) * (2.0 ** -8 if Z.dtype == torch.bfloat16 else F32)
    off = np.abs(np64(gZ) - gw)
    assert np.all(off <= tol), (off - tol).max()
    return loss, stats, gZ, kw


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N, V, K, T", [
    (1, 1, 1, 1.0), (3, 2, 1, 2.0), (5, 7, 3, 1.5), (4, 8, 8, 1.0), (2, 9, 4, 4.0), (7, 255, 16, 2.0), (3, 2047, 64, 0.5),
    (2, 2048, 256, 1.0), (2, 2049, 257, 2.0), (1, 8193, 1024, 1.0), (6, 4096, 1, 8.0), (1300, 33, 5, 2.0), (1100, 2056, 9, 1.5),
    (2, 32000, 64, 2.0), (3, 32003, 33, 1.0), (1, 131071, 100, 2.0), (2, 70000, 1024, 2.0), (1030, 70, 1024, 3.0),
])
def test_against_the_oracle(N, V, K, T, dt):
    run_both(*make(N, V, K, dt, seed=N + V), T=T, w_ce=0.5, w_kd=0.5 * T * T)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_terms_left_out(dt):
    Z, y, ids, t, g = make(6, 300, 12, dt, seed=1)
    run_both(Z, y, None, None, g)
    run_both(Z, None, ids, t, g, T=2.0)
    run_both(Z, y, ids, t, g, w_kd=0.0)
    run_both(Z, y, ids, t, g, w_ce=0.0, T=3.0)
    loss, stats, gZ, _ = run_both(Z, None, None, None, g)
    assert torch.all(loss == 0) and torch.all(gZ == 0)
    run_both(Z, y, ids, t, g, w_ce=-0.5, w_kd=-2.0)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_ids_of_every_kind(dt):
    Z, y, ids, t, g = make(8, 100, 20, dt, seed=2)
    ids[0] = -1                      # no entry
    ids[1] = 7                       # one id twenty times
    ids[2, ::2], y[2] = 50, 50       # an id ten times, the label too
    ids[3] = torch.tensor([100, -5, 2 ** 31 - 1, -2 ** 31] * 5)  # none of them in range
    t[4] = -float("inf")             # no entry either
    t[5, 3:] = -float("inf")
    y[6], y[7] = 100, -2 ** 31       # no label
    loss, stats, gZ, _ = run_both(Z, y, ids, t, g, T=2.0)
    y[0] = y[3] = y[4] = -1
    loss, stats, gZ, _ = run_both(Z, y, ids, t, g, T=2.0)
    assert torch.all(loss[[0, 3, 4]] == 0) and torch.all(gZ[[0, 3, 4]] == 0)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1.0, 2.0])
def test_masked_and_extreme_logits(dt, T):
    # 2500 columns: two slices a row; a masked vocabulary, by -inf and by the type's lowest value
    Z, y, ids, t, g = make(4, 2500, 4, dt, seed=3)
    Z[0, 100:2400] = -float("inf")
    Z[1, 5:] = torch.finfo(DT[dt]).min
    Z[2] = -float("inf")
    Z[2, 2499] = 3.0
    Z[3] *= 60.0
    # a row that is the lowest value throughout: its log-sum is that value in fp32
    low = torch.full((1, 300), torch.finfo(DT[dt]).min, dtype=DT[dt], device=DEV)
    l, st = lac.stage_distill(low, torch.zeros(1, dtype=torch.int32, device=DEV))
    assert torch.isfinite(l).all() and st[0, 0].item() == low[0, 0].item()
    gl = lac.stage_distill_bwd(torch.ones(1, device=DEV), low, st, torch.zeros(1, dtype=torch.int32, device=DEV))
    assert torch.isfinite(gl).all()
    ids[0], y[0] = torch.tensor([1, 2, 2450, 99]), 3
    ids[1], y[1] = torch.tensor([0, 1, 2, 3]), 4
    ids[2], y[2] = 2499, 2499
    loss, stats, gZ, kw = lac.stage_distill(Z, y, ids, t, T), None, None, None
    (loss, stats), n = loss, 3
    zn = np64(Z)
    want, ws, _ = block.distill(zn, y.cpu().numpy(), ids.cpu().numpy(), np64(t), T, 1.0, 1.0)
    assert np.allclose(np64(loss)[:n], want[:n], rtol=2e-5, atol=2e-5) and np.allclose(np64(stats), ws, rtol=1e-5)
    gZ = lac.stage_distill_bwd(g, Z, stats, y, ids, t, T)
    gw, _ = block.distill_bwd(np64(g), zn, y.cpu().numpy(), ids.cpu().numpy(), np64(t), T, 1.0, 1.0)
    # the exponents reach several hundreds in the last row
    assert np.all(np.abs(np64(gZ) - gw) <= (2.0 ** -8 if dt == "bf16" else 1e-4) * np.abs(gw) + 1e-4 * np.abs(np64(g))[:, None])
    # the label or an entry at a logit of -inf: an infinite loss, a finite gradient
    y[0], ids[2, 0] = 200, 0
    loss, stats = lac.stage_distill(Z, y, ids, t, T)
    assert torch.isinf(loss[0]) and torch.isinf(loss[2]) and torch.isfinite(loss[1])
    assert torch.isfinite(lac.stage_distill_bwd(g, Z, stats, y, ids, t, T)).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_do_not_mix(bad):
    Z, y, ids, t, g = make(6, 5000, 10, "bf16", seed=4)
    a = lac.stage_distill(Z, y, ids, t, 2.0)
    ga = lac.stage_distill_bwd(g, Z, a[1], y, ids, t, 2.0)
    Z[3, 4000] = bad
    y[3] = 5
    b = lac.stage_distill(Z, y, ids, t, 2.0)
    gb = lac.stage_distill_bwd(g, Z, b[1], y, ids, t, 2.0)
    keep = [0, 1, 2, 4, 5]
    assert torch.equal(a[0][keep], b[0][keep]) and torch.equal(a[1][keep], b[1][keep]) and torch.equal(ga[keep], gb[keep])
    assert not torch.isfinite(b[0][3])
    # without label and entries a row is 0 whatever its logits
    y[3], ids[3] = -1, -1
    b = lac.stage_distill(Z, y, ids, t, 2.0)
    assert b[0][3] == 0 and torch.all(lac.stage_distill_bwd(g, Z, b[1], y, ids, t, 2.0)[3] == 0)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N, V", [(2, 70001), (1500, 120), (3, 2500), (9, 5)])
def test_in_place_and_repeats(N, V, dt):
    Z, y, ids, t, g = make(N, V, 7, dt, seed=5)
    kw = dict(labels=y, t_ids=ids, t_logits=t, temperature=2.0)
    a, b = lac.stage_distill(Z, **kw), lac.stage_distill(Z, **kw)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    want = lac.stage_distill_bwd(g, Z, a[1], **kw)
    got = lac.stage_distill_bwd(g, Z, a[1], gZ=Z, **kw)
    assert got is Z and torch.equal(got, want)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_at_any_address(dt):
    for V, first in ((64, 1), (65, 1), (2051, 3), (4096, 1)):
        Z, y, ids, t, g = make(3, V, 5, dt, seed=V)
        flat = torch.full((3 * V + 2 * first,), 7.0, dtype=DT[dt], device=DEV)
        Zs = flat[first:first + 3 * V].view(3, V)
        Zs.copy_(Z)
        out = torch.full_like(flat, 7.0)
        run_both(Zs, y, ids, t, g, T=2.0)
        _, stats = lac.stage_distill(Zs, y, ids, t, 2.0)
        lac.stage_distill_bwd(g, Zs, stats, y, ids, t, 2.0, gZ=out[first:first + 3 * V].view(3, V))
        assert torch.all(out[:first] == 7) and torch.all(out[first + 3 * V:] == 7)


def test_leading_axes_streams_graphs_and_errors():
    V = 70000  # two slices a row
    Z, y, ids, t, g = make(6, V, 8, "bf16", seed=6)
    kw = dict(labels=y, t_ids=ids, t_logits=t, temperature=2.0)
    loss, stats = lac.stage_distill(Z, **kw)
    gZ = lac.stage_distill_bwd(g, Z, stats, **kw)
    kw3 = dict(labels=y.view(2, 3), t_ids=ids.view(2, 3, 8), t_logits=t.view(2, 3, 8), temperature=2.0)
    l3, s3 = lac.stage_distill(Z.view(2, 3, V), **kw3)
    g3 = lac.stage_distill_bwd(g.view(2, 3), Z.view(2, 3, V), s3, **kw3)
    assert torch.equal(l3.view(6), loss) and torch.equal(g3.view(6, V), gZ)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    l2, s2 = lac.stage_distill(Z, stream=s, **kw)
    s.synchronize()
    assert torch.equal(l2, loss) and torch.equal(s2, stats)
    ws = torch.empty(lac.stage_distill_workspace_bytes(6, V), dtype=torch.uint8, device=DEV)
    out = [torch.empty_like(x) for x in (loss, stats, gZ)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lac.stage_distill(Z, loss=out[0], stats=out[1], ws=ws, **kw)
        lac.stage_distill_bwd(g, Z, out[1], gZ=out[2], **kw)
    for turn in range(3):
        Z.mul_(0.7)
        for x in out:
            x.zero_()
        want = lac.stage_distill(Z, **kw)
        want += (lac.stage_distill_bwd(g, Z, want[1], **kw),)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), turn
    for call in (lambda: lac.stage_distill(Z, y.long()), lambda: lac.stage_distill(Z, y[:-1]),
                 lambda: lac.stage_distill(Z, y, ids), lambda: lac.stage_distill(Z, y, ids, t.bfloat16()),
                 lambda: lac.stage_distill(Z, y, ids, t[:, :-1]), lambda: lac.stage_distill(Z, y, temperature=0.0),
                 lambda: lac.stage_distill(Z.half(), y), lambda: lac.stage_distill(Z, y, ws=ws[:-16]),
                 lambda: lac.stage_distill_bwd(g, Z, stats[:, :1], y), lambda: lac.stage_distill_bwd(g.double(), Z, stats, y)):
        with pytest.raises(lac.MaplError):
            call()
    assert lac.stage_distill(Z[:0], y[:0])[0].shape == (0,)
