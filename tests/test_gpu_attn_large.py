"""Causal attention with scores and values near the ends of fp32, in both forward
forms (blocks of 32 rows whose waves share the keys, blocks of 128 rows)."""
import numpy as np
import pytest
import torch

import learned_activation_compression_amd as lac

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
F32 = 2.0 ** -24  # half a step, relative
FORMS = [([70, 1, 130], 2, 1), ([1100, 1000], 16, 4)]  # few rows; 272 blocks of 128


def edges(lens):
    return torch.tensor(np.cumsum([0, *lens]), dtype=torch.int32, device=DEV)


def softmax_rows(q, k, v, lens, scale):
    """O and lse in float64, head by head."""
    N, Hq, D = q.shape
    G = Hq // k.shape[1]
    o, lse = torch.zeros(q.shape, dtype=torch.float64, device=DEV), torch.zeros(Hq, N, dtype=torch.float64, device=DEV)
    at = 0
    for n in lens:
        r = slice(at, at + n)
        seen = torch.ones(n, n, dtype=torch.bool, device=DEV).tril()
        for h in range(Hq):
            Q, K, V = (x[r, y].double().contiguous() for x, y in ((q, h), (k, h // G), (v, h // G)))
            s = (scale * (Q @ K.t().contiguous())).masked_fill(~seen, -torch.inf)
            lse[h, r] = torch.logsumexp(s, 1)
            o[r, h] = torch.softmax(s, 1) @ V
        at += n
    return o, lse


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("lens, Hq, Hkv", FORMS)
@pytest.mark.parametrize("D, size, scale", [(64, 8, 2.0 ** 12), (64, 8, 2.0 ** 22), (64, 8, 2.0 ** 28), (64, 8, 2.0 ** 34),
                                            (64, 8, 2.0 ** 64), (80, 8, 2.0 ** 64), (64, 2.0 ** 17, 0.125),
                                            (128, 2.0 ** 22, 0.125)])
def test_scores_of_the_largest_size(D, size, scale, lens, Hq, Hkv, dt):
    # few bits a factor, so that every score is exact: keys of a row's largest score share its
    # weight, and no other, a unit of 2^12 away at least, has any
    g = torch.Generator(device=DEV).manual_seed(D)
    N = sum(lens)
    q, k = ((torch.randint(-8, 9, (N, h, D), generator=g, device=DEV) * (size / 8)).to(DT[dt]) for h in (Hq, Hkv))
    v = torch.randn(N, Hkv, D, generator=g, device=DEV).to(DT[dt])
    k[5], k[lens[0] + 3] = k[0], k[lens[0]]  # and some shared
    want, wlse = softmax_rows(q, k, v, lens, scale)
    O, lse = lac.stage_attn(q, k, v, edges(lens), scale)
    assert torch.isfinite(O).all() and torch.isfinite(lse).all()
    # one key, or a mean of few: the mean's roundings and the output's
    half = 2 * 2.0 ** -8 if dt == "bf16" else 16 * F32
    assert torch.all((O.double() - want).abs() <= half * v.double().abs().max()), (O.double() - want).abs().max()
    # the scale times log2 e, the largest score by it, and back: four roundings, and the output's
    assert torch.all((lse.double() - wlse).abs() <= 6 * F32 * wlse.abs() + 2 * F32)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("lens, Hq, Hkv", FORMS)
@pytest.mark.parametrize("D", [40, 64, 128])
def test_values_near_the_largest(D, lens, Hq, Hkv, dt):
    # a mean of values lies among them, whatever their sum
    g = torch.Generator(device=DEV).manual_seed(D)
    N = sum(lens)
    q = torch.full((N, Hq, D), 1.0, device=DEV).to(DT[dt])
    # scores rise by up to 5 over the sequence: late weights are far above the first
    k = (torch.linspace(0, 5, N, device=DEV)[:, None, None] / D ** 0.5).expand(N, Hkv, D).contiguous().to(DT[dt])
    v = ((0.5 + 0.5 * torch.rand(N, Hkv, D, generator=g, device=DEV)) * 2.0 ** 127).to(DT[dt])
    want, wlse = softmax_rows(q, k, v, lens, D ** -0.5)
    O, lse = lac.stage_attn(q, k, v, edges(lens))
    n, worst = max(lens), 5.1
    # all terms of one sign: the sum of sizes is the output; scores to (D + 4) half steps of theirs
    rel = (2 * (D + 4) * worst + n + 16) * F32 + (2 * 2.0 ** -8 if dt == "bf16" else F32)
    assert torch.isfinite(O).all() and torch.all((O.double() - want).abs() <= rel * want)
    assert torch.all((lse.double() - wlse).abs() <= ((D + 4) * worst + 4 * wlse.abs() + n + 8) * F32)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("lens, Hq, Hkv", FORMS)
@pytest.mark.parametrize("D", [40, 64, 77, 128])
def test_infinities_and_nan_that_rows_see_or_not(D, lens, Hq, Hkv, dt):
    # in the last sequence: column 3 is infinite from a key on, and again, with the other sign, behind a
    # later one; column 5 is NaN from a third on; the last key, that its own row alone sees, is
    # spoilt in every column of another kind.  The other columns and rows are as without
    g = torch.Generator(device=DEV).manual_seed(D)
    N, n = sum(lens), lens[-1]
    first = N - n
    q, k, v = (torch.randn(N, h, D, generator=g, device=DEV).to(DT[dt]) for h in (Hq, Hkv, Hkv))
    clean, clse = lac.stage_attn(q, k, v, edges(lens))
    a, b, c = first + 9, first + n // 2, first + n // 2 + 40
    v[a, :, 3], v[b, :, 3], v[c, :, 5] = float("inf"), -float("inf"), float("nan")
    v[N - 1, :, ::2], v[N - 1, :, 1::2] = float("nan"), float("inf")
    O, lse = lac.stage_attn(q, k, v, edges(lens))
    assert torch.equal(lse, clse)
    row = torch.arange(N, device=DEV)
    spoilt = torch.zeros(O.shape, dtype=torch.bool, device=DEV)
    assert torch.all(O[(row >= a) & (row < b), :, 3] == float("inf")) and torch.isnan(O[b:, :, 3]).all()
    assert torch.isnan(O[c:, :, 5]).all() and not torch.isfinite(O[N - 1]).any()
    spoilt[a:, :, 3], spoilt[c:, :, 5], spoilt[N - 1] = True, True, True
    # a row formed again adds up in another order, and its weights are not rounded to bf16
    tol = 2.0 ** -6 if dt == "bf16" else 1e-5
    off = (O.float() - clean.float()).abs()
    assert torch.isfinite(O[~spoilt]).all() and torch.all(off[~spoilt] <= tol * (1 + clean[~spoilt].float().abs()))
