"""The example's training step around the boundary: every activation and
gradient of its forward and backward pass against the same step composed in
float64 from the oracles, each operator fed with what the GPU step fed it."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import codec, stage
from parity_util import BF16_TOL, np64, rel_l2

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("stage_boundary", os.path.join(ROOT, "examples", "stage_boundary.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _t(x):
    return np.ascontiguousarray(x.T)


def test_training_step_around_the_boundary():
    ex = _example()
    N, d, r, drop, seed, row = 300, 256, 64, 0.1, 99, (1 << 32) - 7
    dev = ex.make(N, d, r, vocab=50)
    out = {k: np64(v) for k, v in ex.step(dev, drop, seed, row).items()}
    p = {k: np64(v) for k, v in dev.items()}
    t = dev["tids"].cpu().numpy()
    rows, square = stage.round_blocks, lambda w: stage.round_blocks(w, square=True)
    kw = dict(res_scale=0.8, eps=1e-5, p=drop, seed=seed, offset=row)

    ref = {"y": rows(p["a"]) @ square(p["W_out"]).T}
    ref["X"], _ = stage.norm(p["x"], out["y"], p["w_post"], p["gate"], **kw)
    ref["Z"] = codec.compress(out["X"], t, p["E"], p["P"], p["A"])
    ref["Xhat"] = codec.reconstruct(out["Z"], t, p["E"], p["P"], p["A"])
    _, ref["h"] = stage.norm(out["Xhat"], w_pre=p["w_pre"])
    ref["q"] = stage.dropout(rows(out["h"]) @ square(p["W_in"]).T, drop, seed + 1, row)
    ref["gz"] = stage.dropout(p["gq"], drop, seed + 1, row)
    ref["gh"] = rows(out["gz"]) @ square(p["W_in"])
    ref["gW_in"] = rows(_t(out["gz"])) @ rows(_t(out["h"])).T
    b = stage.norm_bwd(None, out["gh"], out["Xhat"], None, None, None, p["w_pre"], 1.0, 1e-5, 0.0, 0, 0)
    ref.update(gXhat=b["gX"], g_w_pre=b["g_w_pre"])
    ref["gZ"], gA = codec.reconstruct_bwd(out["gXhat"], out["Z"], p["A"])
    ref["gX"], gA2 = codec.compress_bwd(out["gZ"], out["X"], t, p["E"], p["P"], p["A"])
    ref["gA"] = gA + gA2
    b = stage.norm_bwd(out["gX"], None, None, out["y"], p["w_post"], p["gate"], None, *kw.values())
    ref.update(gx=b["gX"], gy=b["gY"], g_w_post=b["g_w_post"], g_gate=b["g_gate"])
    ref["ga"] = rows(out["gy"]) @ square(p["W_out"])
    ref["gW_out"] = rows(_t(out["gy"])) @ rows(_t(p["a"])).T
    for k, v in ref.items():
        assert rel_l2(out[k], v) <= BF16_TOL, (k, rel_l2(out[k], v))
    assert set(out) == set(ref)


def test_the_step_repeats_bitwise_and_splits_by_rows():
    ex = _example()
    dev = ex.make(256, 256, 64, vocab=50, seed=3)
    a, b = ex.step(dev, 0.2, 5, 100), ex.step(dev, 0.2, 5, 100)
    for k in a:
        assert torch.equal(a[k], b[k]), k
    # the second half of the tokens as a micro-batch of its own, its rows counted on: the same activations
    half = {k: v[128:] if v.shape[0] == 256 and k in ("x", "a", "gq", "tids") else v for k, v in dev.items()}
    c = ex.step({k: v.contiguous() for k, v in half.items()}, 0.2, 5, 228)
    for k in ("y", "X", "Z", "Xhat", "h", "q", "gx", "ga"):
        assert rel_l2(np64(c[k]), np64(a[k][128:])) <= BF16_TOL, k
