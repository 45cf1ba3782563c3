"""Backward of the block edge in the forms that leave most of it out: gX_out
alone (no block output, no gradient of H), whose gradient is gX = res_scale
gX_out."""
import pytest
import torch

import learned_activation_compression_amd as lac

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N, d", [(1, 1), (3, 7), (5, 8), (33, 129), (7, 1003), (300, 1024), (9, 5000), (4, 8192)])
def test_gradient_of_the_scaled_residual_alone(N, d, dt):
    g = torch.Generator(device=DEV).manual_seed(N + d)
    gx = torch.randn(N, d, device=DEV, generator=g).to(DT[dt])
    # one product in fp32, rounded once: the same value in torch
    want = (torch.tensor(0.7, device=DEV) * gx.float()).to(DT[dt])
    out = lac.stage_norm_bwd(gx, res_scale=0.7)
    assert torch.equal(out[0], want) and out[1:] == (None, None, None, None)
    # what only the gradient of H would read may be there all the same
    x, w = torch.full_like(gx, float("nan")), torch.ones(d, dtype=DT[dt], device=DEV)
    assert torch.equal(lac.stage_norm_bwd(gx, X_out=x, w_pre=w, res_scale=0.7)[0], want)
    # over gX_out itself, and between guard values at an odd offset
    buf = torch.full((N * d + 64,), 5.0, dtype=DT[dt], device=DEV)
    at = buf[17:17 + N * d].view(N, d)
    lac.stage_norm_bwd(gx, res_scale=0.7, gX=at)
    assert torch.equal(at, want) and (buf[:17] == 5).all() and (buf[17 + N * d:] == 5).all()
    assert lac.stage_norm_bwd(gx, res_scale=0.7, gX=gx)[0] is gx and torch.equal(gx, want)


def test_gradient_of_the_scaled_residual_of_no_rows():
    gx = torch.empty(0, 64, device=DEV)
    assert lac.stage_norm_bwd(gx)[0].shape == (0, 64)
