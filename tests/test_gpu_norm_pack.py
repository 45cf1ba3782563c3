"""The block edge with an 8-bit output against its two parts: X_out and H are
stage_norm's but for the rounding of its fp32 sums (here they are fp64), and the pack
is that of H before rounding."""
import numpy as np
import pytest
import torch

import learned_activation_compression_amd as lac
from oracle import stage

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
WIDTHS = [1, 7, 8, 64, 127, 128, 129, 200, 256, 500, 512, 1000, 1024, 1023, 1536, 2048, 2047, 4096, 5000, 8192]


def make(N, d, dt, G, seed=0, post=True, y=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    f = lambda x: x.to(DEV, DT[dt])  # noqa: E731
    ch = torch.exp(0.5 * r(d))
    return dict(X=f(r(N, d) * ch), Y=f(r(N, d) * ch) if y else None, w_post=f(1 + 0.2 * r(d)) if y and post else None,
                gate=f(0.5 + 0.2 * r(G, d)) if y and G else None, w_pre=f(1 + 0.2 * r(d)))


def values(pk, N, d):
    return lac.fp8_unpack(pk, N, d)


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("N, G, p, y", [(1, 1, 0.0, True), (33, 1, 0.2, True), (70, 70, 0.0, True), (64, 0, 0.1, True),
                                        (41, 0, 0.0, False)])
def test_fp32_is_its_two_parts(N, G, p, y, d):
    # in fp32 H is not rounded: the pack is that of the stored H, bit for bit
    a = make(N, d, "f32", G, seed=d + N, y=y)
    kw = dict(res_scale=0.8, p=p, seed=5, offset=9)
    X_out, H = lac.stage_norm(**a, **kw)
    x, h, pk = lac.stage_norm_pack(**a, **kw, store_h=True)
    # stage_norm's sum of squares is a chain of at most 8 (two vectors: 16) + 6 + 16 additions,
    # so that its root is off by up to 19 half steps; the products and sums add 5 to that
    size = 0.8 * a["X"].abs() + (X_out - 0.8 * a["X"]).abs()
    assert torch.all((x - X_out).abs() <= 24 * 2.0 ** -24 * size)
    scale = (H / X_out).abs().nan_to_num(posinf=0.0)
    assert torch.all((h - H).abs() <= 2.0 ** -24 * (24 * H.abs() + 24 * scale * size))
    want, _ = lac.fp8_pack(h)
    assert torch.equal(values(pk, N, d), values(want, N, d))
    n, none, pk2 = lac.stage_norm_pack(**a, **kw, store_x=False)
    assert n is None and none is None and torch.equal(values(pk2, N, d), values(want, N, d))


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("N, G", [(1, 1), (50, 1), (65, 5)])
def test_bf16_rounds_once(N, G, d):
    # the same numbers in fp32 give H unrounded (the weights' and the inputs' values are bf16's)
    a = make(N, d, "bf16", G, seed=d)
    X_out, H = lac.stage_norm(**a, res_scale=0.8)
    x, h, pk = lac.stage_norm_pack(**a, res_scale=0.8, store_h=True)
    # numbers that differ in their last fp32 bits round to the same or to neighbours; small
    # sums of large terms may differ by those terms' last bits
    for got, want, top in ((x, X_out, a["X"]), (h, H, H)):
        assert torch.all((got.float() - want.float()).abs() <= 2.0 ** -7 * want.float().abs() + 2.0 ** -20 * top.float().abs().max())
        assert (got != want).float().mean() <= 1e-3 or (got != want).sum() <= 1
    _, H32 = lac.stage_norm(**{k: v.float() for k, v in a.items()}, res_scale=0.8)
    want = values(lac.fp8_pack(H32)[0], N, d)
    got = values(pk, N, d)
    # the two forms may add up in another order where a row is split differently over lanes
    off = (got != want).float().mean().item()
    assert off <= 1e-4 or off * N * d <= 2
    assert torch.all((got - want).abs() <= 2.0 ** -3 * want.abs() + 2.0 ** -8 * want.abs().max())


def test_pack_against_the_oracle():
    a = make(40, 300, "f32", 1, seed=3)
    n = {k: v.cpu().double().numpy() for k, v in a.items()}
    _, h = stage.norm(n["X"], n["Y"], n["w_post"], n["gate"], n["w_pre"], 0.8, 1e-5)
    _, _, pk = lac.stage_norm_pack(**a, res_scale=0.8)
    got, want = values(pk, 40, 300).cpu().double().numpy(), stage.round_blocks(h)
    # half a step of e4m3 (2^-4) of the value, half the smallest code of its block (2^-10 of its scale), and fp32
    top = np.abs(h).reshape(40, -1).max()
    assert np.all(np.abs(got - h) <= (2.0 ** -4 + 1e-5) * np.abs(h) + 2.0 ** -10 * top / 224)
    assert np.mean(got != want) <= 1e-3


def test_products_take_the_pack():
    N, d, M = 100, 384, 256
    a = make(N, d, "bf16", 1, seed=8)
    W = torch.randn(M, d, device=DEV).to(torch.bfloat16)
    W8, _ = lac.fp8_pack(W, square=True)
    _, _, pk = lac.stage_norm_pack(**a)
    Y = lac.fp8_gemm(pk, W8, N, M, d, dtype=torch.float32)
    want = values(pk, N, d).double() @ values(W8, M, d).double().t()
    size = values(pk, N, d).double().abs() @ values(W8, M, d).double().abs().t()
    assert torch.all((Y.double() - want).abs() <= d * 2.0 ** -24 * size)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_values_that_are_not_finite(dt):
    a = make(40, 300, dt, 0, seed=4)
    a["X"][3, 5] = float("nan")
    a["X"][4] = 0
    a["Y"][4] = 0
    a["w_pre"][200] = float("inf")
    x, h, pk = lac.stage_norm_pack(**a, store_h=True)
    got = values(pk, 40, 300)
    assert torch.equal(torch.isnan(got), ~torch.isfinite(h))
    assert torch.isnan(got[3]).all() and torch.all(got[4, :200] == 0)
    want = values(lac.fp8_pack(h)[0], 40, 300)
    ok = torch.isfinite(got)
    assert torch.all((got[ok] - want[ok]).abs() <= 2.0 ** -3 * want[ok].abs() + 2.0 ** -7)


def test_padding_streams_graphs_and_errors():
    N, d = 40, 200
    a = make(N, d, "bf16", 1, seed=6)
    n = lac.fp8_pack_bytes(N, d)
    # a pack of NaN codes before the call: padding columns become zero, so that products with it are finite
    pk = torch.full((n,), 0x7F, dtype=torch.uint8, device=DEV)
    x, _, got = lac.stage_norm_pack(**a, pkH=pk)
    assert got is pk
    W8, _ = lac.fp8_pack(torch.ones(16, d, device=DEV), square=True)
    assert torch.isfinite(lac.fp8_gemm(pk, W8, N, 16, d)).all()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    x2, _, pk2 = lac.stage_norm_pack(**a, stream=s)
    s.synchronize()
    assert torch.equal(x, x2) and torch.equal(values(pk, N, d), values(pk2, N, d))
    out, pkg = torch.empty_like(x), torch.empty_like(pk)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lac.stage_norm_pack(**a, X_out=out, pkH=pkg)
    for _ in range(3):
        a["X"].mul_(0.5)
        want = lac.stage_norm_pack(**a)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(values(pkg, N, d), values(want[2], N, d))
    for kw in (dict(w_pre=None), dict(w_pre=a["w_pre"].float()), dict(pkH=pk[:-1]), dict(eps=0.0), dict(Y=a["Y"][:-1])):
        with pytest.raises(lac.MaplError):
            lac.stage_norm_pack(**{**a, **kw})
    assert lac.stage_norm_pack(a["X"][:0], w_pre=a["w_pre"])[0].shape == (0, d)


@pytest.mark.parametrize("N, d", [(1, 128), (33, 200), (40, 1024), (70, 2048), (31, 4100)])
def test_the_pack_is_the_same_bytes(N, d):
    # fp8_pack's, with the zeros behind the last row and column; exponents of whole units of 32 rows
    a = make(N, d, "f32", 1, seed=N)
    n = lac.fp8_pack_bytes(N, d)
    pk = [torch.full((n,), 0x7F, dtype=torch.uint8, device=DEV) for _ in range(2)]
    _, h, _ = lac.stage_norm_pack(**a, store_h=True, pkH=pk[0])
    lac.fp8_pack(h, pk=pk[1])
    assert torch.equal(pk[0], pk[1])
