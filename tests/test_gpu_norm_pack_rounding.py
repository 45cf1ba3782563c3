"""One rounding from the exact value to the bf16 outputs and the 8-bit codes of the
block edge, on inputs whose norms are exact: rows of small whole numbers."""
import pytest
import torch

import learned_activation_compression_amd as lac

pytestmark = pytest.mark.gpu
DEV = "cuda"


def pow2(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def e4m3(x):
    """float64 [N][d], d a multiple of 128, on the grid of each row's blocks of 128 columns."""
    v = x.view(x.shape[0], -1, 128)
    top = v.abs().amax(2, keepdim=True)
    m, e = torch.frexp(top)
    unit = pow2(e - 9 + (m > 0.875).int())
    _, e = torch.frexp(v / unit)
    ulp = unit * pow2(torch.clamp(e - 1, min=-6) - 3)
    return (torch.round(v / ulp) * ulp).view(x.shape)


def bf16(x):
    """float64 to bf16 in one rounding: the 45 bits below its 8, none of the values near 2^-126."""
    b = x.view(torch.int64)
    b = b + ((1 << 44) - 1) + ((b >> 45) & 1)
    return (b >> 45 << 45).view(torch.float64).to(torch.bfloat16)


def test_the_rounding_itself():
    x = torch.tensor([1.0, 1 + 2.0 ** -8, 1 + 2.0 ** -8 + 2.0 ** -40, 1 + 3 * 2.0 ** -8, -1 - 2.0 ** -8 - 2.0 ** -40],
                     dtype=torch.float64)
    assert bf16(x).tolist() == [1.0, 1.0, 1 + 2.0 ** -7, 1 + 2.0 ** -6, -1 - 2.0 ** -7]


@pytest.mark.parametrize("N, d", [(16384, 1024), (2048, 8192)])
@pytest.mark.parametrize("edge", [False, True])
def test_one_rounding(edge, N, d):
    # 16 million elements: some hundreds lie so close to the middle of two bf16 numbers, and
    # some ten to that of two codes, that a rounding to fp32 on the way would put them there
    g = torch.Generator(device=DEV).manual_seed(d + edge)
    whole = lambda *s: torch.randint(-90, 91, s, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    weight = lambda *s: (1 + 0.2 * torch.randn(s, generator=g, device=DEV)).to(torch.bfloat16)  # noqa: E731
    X, w_pre = whole(N, d), weight(d)
    if edge:
        Y, w_post, gate = whole(N, d), weight(d), weight(1, d)
        out, _, _ = lac.stage_norm_pack(X, Y, w_post, gate, w_pre, res_scale=0.75, eps=2.0 ** -10)
        y = Y.double()
        # the mean of squares is exact, and so are the products of three bf16 numbers
        x = 0.75 * X.double()
        v = torch.rsqrt((y * y).mean(1, keepdim=True) + 2.0 ** -10) * (y * w_post.double() * gate.double())
        want, size = x + v, x.abs() + v.abs()
        # what a few roundings of float64 decide is left out
        near = [bf16(want + s * 2.0 ** -48 * size) for s in (-1, 1)]
        sure = near[0] == near[1]
        assert sure.float().mean() > 0.99 and torch.equal(out[sure], bf16(want)[sure])
        return
    _, H, pk = lac.stage_norm_pack(X, w_pre=w_pre, eps=2.0 ** -10, store_x=False, store_h=True)
    x = X.double()
    want = x * torch.rsqrt((x * x).mean(1, keepdim=True) + 2.0 ** -10) * w_pre.double()
    near = [bf16(want * (1 + s * 2.0 ** -48)) for s in (-1, 1)]
    sure = near[0] == near[1]
    assert torch.equal(H[sure], bf16(want)[sure])
    near = [e4m3(want * (1 + s * 2.0 ** -48)) for s in (-1, 1)]
    sure = near[0] == near[1]
    got = lac.fp8_unpack(pk, N, d).double()
    off = (got != e4m3(want)) & sure
    assert not off.any(), (off.sum().item(), want[off][:4], got[off][:4], e4m3(want)[off][:4])
