"""Calls of the stage operators that leave most arguments out, without a GPU:
what the C ABI takes and refuses before anything is enqueued."""
import ctypes

import pytest
import torch

import learned_activation_compression_amd as lac
from learned_activation_compression_amd import stage as binding

ENULL, EARG, EHIP = -1, -4, -6
FAKE = ctypes.c_void_p(0x1000)  # never dereferenced


@pytest.mark.skipif(torch.cuda.is_available(), reason="a device is present: valid calls would launch kernels")
@pytest.mark.parametrize("dt", [lac.MAPL_BF16, lac.MAPL_F32])
def test_backward_of_the_scaled_residual_alone(dt):
    lib = binding._stage_lib()

    def bwd(gX_out=FAKE, gH=None, X_out=None, Y=None, w_pre=None, gX=FAKE, g_w_pre=None, p=0.0, ws=None):
        return lib.stage_norm_bwd(gX_out, gH, X_out, Y, None, None, w_pre, gX, None, None, None, g_w_pre, 0, 0.5, 1e-5, p,
                                  0, 0, 4, 64, 0, dt, ws, 0, None)

    assert bwd() == EHIP  # taken: the device set-up's error
    assert bwd(X_out=FAKE, w_pre=FAKE) == EHIP
    assert bwd(gX=None) == ENULL and bwd(gX_out=None) == ENULL and bwd(p=0.1) == EARG
    # with a gradient of H each of its tensors is needed
    assert bwd(gH=FAKE) == ENULL and bwd(gH=FAKE, w_pre=FAKE, g_w_pre=FAKE) == ENULL
    assert bwd(gH=FAKE, X_out=FAKE, w_pre=FAKE, g_w_pre=FAKE) == ENULL  # no workspace


def test_a_stream_of_another_device_is_refused():
    # entering it would leave the tensors' device, and the call would then run on that device's current stream instead
    from types import SimpleNamespace
    like = SimpleNamespace(device=torch.device("cuda", 0))
    with pytest.raises(lac.MaplError) as e:
        with binding._there(like, SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)):
            pass
    assert e.value.status == -1 and "cuda:1" in str(e.value) and "cuda:0" in str(e.value)
