"""Causal attention at the edges of its inputs' range, in both forward forms (blocks
of 32 rows whose waves share the keys, blocks of 128 rows): visible infinities at head
widths that are padded."""
import numpy as np
import pytest
import torch

import learned_activation_compression_amd as lac

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
F32 = 2.0 ** -24  # half a step, relative
FORMS = [([70, 130], 2, 1), ([1100, 1000], 16, 4)]  # few rows; 272 blocks of 128


def edges(lens):
    return torch.tensor(np.cumsum([0, *lens]), dtype=torch.int32, device=DEV)


def reference(q, k, v, go, lens, scale, gone):
    """O, lse, gradients and sizes in float64, sequence by sequence and head by head, where no row
    sees the keys `gone` (of weight 0)."""
    N, Hq, D = q.shape
    G = Hq // k.shape[1]
    out = {n: torch.zeros(s, dtype=torch.float64, device=DEV) for n, s in
           (("o", q.shape), ("gq", q.shape), ("gk", k.shape), ("gv", v.shape), ("lse", (Hq, N)))}
    size = {n: torch.zeros_like(x) for n, x in out.items()}
    at = 0
    for n in lens:
        r = slice(at, at + n)
        seen = torch.ones(n, n, dtype=torch.bool, device=DEV).tril()
        seen[:, [j - at for j in gone if at <= j < at + n]] = False
        for h in range(Hq):
            Q, K, V, g = (x[r, y].double().contiguous() for x, y in ((q, h), (k, h // G), (v, h // G), (go, h)))
            s = (scale * (Q @ K.t().contiguous())).masked_fill(~seen, -torch.inf)
            lse = torch.logsumexp(s, 1, keepdim=True)
            p = torch.exp(s - lse)
            o = p @ V
            delta = (g * o).sum(1, keepdim=True)
            ds = scale * p * (g @ V.t().contiguous() - delta)
            dz = scale * p * (g.abs() @ V.abs().t().contiguous() + (g * o).abs().sum(1, keepdim=True))
            out["o"][r, h], out["lse"][h, r], out["gq"][r, h] = o, lse[:, 0], ds @ K
            size["o"][r, h], size["gq"][r, h] = p @ V.abs(), dz @ K.abs()
            size["lse"][h, r] = (scale * (Q.abs() @ K.abs().t().contiguous())).masked_fill(~seen, 0).amax(1)
            out["gk"][r, h // G] += ds.t().contiguous() @ Q
            out["gv"][r, h // G] += p.t().contiguous() @ g
            size["gk"][r, h // G] += dz.t().contiguous() @ Q.abs()
            size["gv"][r, h // G] += p.t().contiguous() @ g.abs()
        at += n
    return out, size


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("lens, Hq, Hkv", FORMS)
@pytest.mark.parametrize("D", [8, 32, 40, 64, 80, 112, 128])
def test_a_visible_score_of_minus_infinity(D, lens, Hq, Hkv, dt):
    # one key is -inf in its first column, where every query is positive: its score is -inf,
    # its weight 0, and the rows that see it are finite, their log-sums too
    g = torch.Generator(device=DEV).manual_seed(D)
    N, j = sum(lens), lens[0] + 7
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    q, k, v, go = r(N, Hq, D), r(N, Hkv, D), r(N, Hkv, D), r(N, Hq, D)
    q[:, :, 0] = q[:, :, 0].abs() + 0.25
    q, k, v, go = (x.to(DT[dt]) for x in (q, k, v, go))
    clean = k.clone()
    clean[j] = 0
    k[j, :, 0] = -float("inf")
    cu, scale = edges(lens), D ** -0.5
    want, size = reference(q, clean, v, go, lens, scale, [j])
    O, lse = lac.stage_attn(q, k, v, cu)
    got = dict(zip(("gq", "gk", "gv"), lac.stage_attn_bwd(go, q, k, v, O, lse, cu)), o=O)
    # as in the tests of finite scores: a score is off by (D + 4) half steps of its products'
    # sizes, a weight by twice that and the log-sum's rounding, sums over n keys by n + 16
    worst, n = size["lse"].max().item(), max(lens)
    ltol = ((D + 4) * 1.01 * size["lse"] + 4 * want["lse"].abs() + n + 8) * F32
    assert torch.isfinite(lse).all() and torch.all((lse.double() - want["lse"]).abs() <= ltol)
    half = 2.0 ** -8 if dt == "bf16" else 0.0
    fwd = (2 * (D + 4) * worst + n + 8) * F32
    bwd = (2 * (D + 4) * worst + 4 * want["lse"].abs().max().item() + 2 * D + n * (Hq // Hkv) + 16) * F32
    bwd += 2.0 ** -8 if dt == "bf16" else F32  # delta from the stored O
    sees = torch.zeros(N, dtype=torch.bool, device=DEV)
    sees[j:] = True
    for name, x in got.items():
        tol = size[name] * ((fwd if name == "o" else bwd) + half) + want[name].abs() * (half + F32) + 1e-30
        ok = torch.ones_like(x, dtype=torch.bool)
        if name == "gq":  # 0 times -inf, in the formula as well
            ok[sees, :, 0] = False
            assert torch.isnan(x[~ok]).all()
        if name in ("gk", "gv"):
            assert torch.all(x[j] == 0), name  # nobody gives it weight
        off = (x.double() - want[name]).abs()
        assert torch.isfinite(x[ok]).all() and torch.all(off[ok] <= tol[ok]), (name, (off - tol)[ok].max().item())
