"""Offsets beyond 32 bits: attention, the loss and the edge with an 8-bit output on
tensors of more than 2^31 elements or 2^32 bytes, against the same rows by themselves,
bit for bit."""
import pytest
import torch

import learned_activation_compression_amd as lac

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dt, ld, N, Hq, Hkv, D", [
    (torch.bfloat16, 1 << 20, 2500, 4, 2, 64),     # few rows at a time, split gradients
    (torch.bfloat16, 1 << 18, 9000, 16, 16, 64),   # blocks of 128 rows
    (torch.float32, 1 << 22, 300, 2, 1, 128),      # the widest rows
])
def test_attention_rows_far_apart(dt, ld, N, Hq, Hkv, D):
    g = torch.Generator(device=DEV).manual_seed(N)
    wide = (2 * Hq + 2 * Hkv) * D
    small = torch.randn(N, wide, generator=g, device=DEV).to(dt)
    far = torch.empty(N, ld, dtype=dt, device=DEV)
    far[:, -wide:] = small
    cu = torch.tensor([0, 200, N // 2, N], dtype=torch.int32, device=DEV)
    cols = [Hq * D, Hkv * D, Hkv * D, Hq * D]
    views = lambda x: [y.unflatten(1, (-1, D)) for y in x[:, -wide:].split(cols, dim=1)]  # noqa: E731
    want, got = views(small), views(far)
    O, lse = lac.stage_attn(*want[:3], cu)
    grads = lac.stage_attn_bwd(want[3], *want[:3], O, lse, cu)
    O2, lse2 = lac.stage_attn(*got[:3], cu)
    assert torch.equal(O, O2) and torch.equal(lse, lse2)
    # the gradients over the inputs' columns of a second tensor, O into it as well
    out = torch.empty(N, ld, dtype=dt, device=DEV)
    gq, gk, gv, o = views(out)
    lac.stage_attn(*got[:3], cu, O=o)
    lac.stage_attn_bwd(got[3], *got[:3], o, lse2, cu, gQ=gq, gK=gk, gV=gv)
    assert torch.equal(o, O) and all(torch.equal(x, y) for x, y in zip((gq, gk, gv), grads))


def test_loss_of_many_rows():
    N, V, K, last = 70000, 32000, 8, 2000
    g = torch.Generator(device=DEV).manual_seed(3)
    base = (3 * torch.randn(last, V, generator=g, device=DEV)).to(torch.bfloat16)
    Z = torch.empty(N, V, dtype=torch.bfloat16, device=DEV)
    for n in range(0, N, last):
        Z[n:n + last] = base
    y = torch.randint(0, V, (N,), generator=g, device=DEV, dtype=torch.int32)
    ids = torch.randint(0, V, (N, K), generator=g, device=DEV, dtype=torch.int32)
    t = torch.randn(N, K, generator=g, device=DEV)
    go = torch.rand(N, generator=g, device=DEV)
    loss, stats = lac.stage_distill(Z, y, ids, t, 2.0, 0.5, 0.5)
    e = slice(N - last, N)
    want, wstats = lac.stage_distill(base, y[e], ids[e], t[e], 2.0, 0.5, 0.5)
    assert torch.equal(loss[e], want) and torch.equal(stats[e], wstats)
    wg = lac.stage_distill_bwd(go[e], base, wstats, y[e], ids[e], t[e], 2.0, 0.5, 0.5)
    gz = lac.stage_distill_bwd(go, Z, stats, y, ids, t, 2.0, 0.5, 0.5, gZ=Z)
    assert torch.equal(gz[e], wg)


def test_edge_of_many_rows():
    N, d, last = 2200000, 1024, 4096
    g = torch.Generator(device=DEV).manual_seed(5)
    X = torch.randn(last, d, generator=g, device=DEV).to(torch.bfloat16).repeat(N // last + 1, 1)[:N]
    w = torch.rand(d, generator=g, device=DEV).to(torch.bfloat16)
    _, _, pk = lac.stage_norm_pack(X, w_pre=w, store_x=False)
    rows = N // 32 * 32 - last  # whole units of 32 rows
    tail = X[rows:].contiguous()
    _, _, want = lac.stage_norm_pack(tail, w_pre=w, store_x=False)
    n = (len(tail) + 31) // 32 * 4096 * (d // 128)
    at = rows // 32 * 4096 * (d // 128)
    assert torch.equal(pk[at:at + n], want[:n])
