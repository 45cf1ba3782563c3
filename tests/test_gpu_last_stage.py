"""The example's training step of a last stage: every activation and gradient of
its forward and backward pass against the same step composed in float64 from the
oracles, each operator fed with what the GPU step fed it."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import block, stage
from parity_util import BF16_TOL, np64, rel_l2

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("last_stage", os.path.join(ROOT, "examples", "last_stage.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _t(x):
    return np.ascontiguousarray(x.T)


def test_training_step_of_the_last_stage():
    ex = _example()
    lens, d, H, G, V, T = [70, 1, 45, 84], 256, 4, 2, 301, 2.0
    D, wide = d // H, (H + 2 * G) * (d // H)
    dev = ex.make(lens, d, H, G, V, 9)
    out = {k: np64(v) for k, v in ex.step(dev, H, G, T).items()}
    p = {k: np64(v) for k, v in dev.items()}
    cu, labels, ids = (dev[k].cpu().numpy() for k in ("cu", "labels", "t_ids"))
    rows, square = stage.round_blocks, lambda w: stage.round_blocks(w, square=True)

    def split(x):
        return (x[:, :H * D].reshape(-1, H, D), x[:, H * D:(H + G) * D].reshape(-1, G, D), x[:, (H + G) * D:].reshape(-1, G, D))

    ref = {}
    _, h = stage.norm(p["Xhat"], w_pre=p["w_1"])
    ref["h"], ref["qkv"] = h, rows(h) @ square(p["W_qkv"]).T
    q, k, v = split(out["qkv"])
    o, ref["lse"], _, _ = block.attn(q, k, v, cu, D ** -0.5)
    ref["o"] = o.reshape(-1, d)
    ref["y"] = rows(out["o"]) @ square(p["W_o"]).T
    ref["X"], f = stage.norm(p["Xhat"], out["y"], p["w_p"], p["gate"], p["w_2"], 0.8)
    ref["f"], ref["z"] = f, rows(f) @ square(p["W_v"]).T
    args = (labels, ids, p["t_logits"], T, 0.5, 0.5 * T * T)
    ref["loss"] = block.distill(out["z"], *args)[0]
    ref["gz"] = block.distill_bwd(p["gloss"], out["z"], *args)[0]
    ref["gf"] = rows(out["gz"]) @ square(p["W_v"])
    ref["gW_v"] = rows(_t(out["gz"])) @ rows(_t(out["f"])).T
    b = stage.norm_bwd(None, out["gf"], out["X"], out["y"], p["w_p"], p["gate"], p["w_2"], 0.8, 1e-5, 0.0, 0, 0)
    ref.update(gx=b["gX"], gy=b["gY"], g_w_p=b["g_w_post"], g_gate=b["g_gate"], g_w_2=b["g_w_pre"])
    ref["go"] = rows(out["gy"]) @ square(p["W_o"])
    ref["gW_o"] = rows(_t(out["gy"])) @ rows(_t(out["o"])).T
    g, _ = block.attn_bwd(out["go"].reshape(-1, H, D), q, k, v, out["o"].reshape(-1, H, D), out["lse"], cu, D ** -0.5)
    ref["gqkv"] = np.concatenate([g[n].reshape(len(q), -1) for n in ("gq", "gk", "gv")], axis=1)
    ref["gh"] = rows(out["gqkv"]) @ square(p["W_qkv"])
    ref["gW_qkv"] = rows(_t(out["gqkv"])) @ rows(_t(out["h"])).T
    b = stage.norm_bwd(out["gx"], out["gh"], p["Xhat"], None, None, None, p["w_1"], 1.0, 1e-5, 0.0, 0, 0)
    ref.update(gXhat=b["gX"], g_w_1=b["g_w_pre"])
    for name, want in ref.items():
        assert rel_l2(out[name], want) <= BF16_TOL, (name, rel_l2(out[name], want))
    assert set(out) == set(ref) and out["gqkv"].shape == (sum(lens), wide)


def test_the_step_repeats_bitwise_and_keeps_sequences_apart():
    ex = _example()
    lens = [50, 30, 100]
    dev = ex.make(lens, 256, 4, 1, 200, 5, seed=3)
    a, b = ex.step(dev, 4, 1), ex.step(dev, 4, 1)
    for k in a:
        assert torch.equal(a[k], b[k]), k
    # the last sequence as a micro-batch of its own: the same activations and row gradients
    one = {k: v[80:].contiguous() if v.shape[0] == 180 else v for k, v in dev.items()}
    one["cu"] = torch.tensor([0, 100], dtype=torch.int32, device="cuda")
    c = ex.step(one, 4, 1)
    for k in ("h", "qkv", "o", "y", "X", "f", "z", "loss", "gz", "gx", "gXhat"):
        assert rel_l2(np64(c[k]), np64(a[k][80:])) <= BF16_TOL, k
