"""The block edge on tensors at any address of their type, between guard values:
every form of row access (vec8.h), each tensor shifted alone and all together.
Tolerances as in test_gpu_stage_norm."""
import numpy as np
import pytest
import torch

import learned_activation_compression_amd as lac
from oracle import stage
from test_gpu_stage_norm import DT, n64, near, rows, steps, vec

pytestmark = pytest.mark.gpu
DEV = "cuda"
GUARD = 5.0
# widths by form: below 8; whole vectors; even; odd; several vectors a thread; slots of several waves
WIDTHS = [3, 6, 8, 64, 130, 131, 1000, 1003, 1026, 1544, 2049, 4099, 4104, 8190]


class Shifted:
    """Copies and empty tensors that start `by` elements into a guarded buffer."""

    def __init__(self, by):
        self.by, self.made = by, []

    def empty(self, shape, dtype):
        n = int(np.prod(shape))
        buf = torch.full((n + 64,), GUARD, dtype=dtype, device=DEV)
        at = 16 + self.by
        self.made.append((buf, at, at + n))
        return buf[at:at + n].view(shape)

    def copy(self, t):
        return self.empty(t.shape, t.dtype).copy_(t)

    def check(self, what):
        for buf, lo, hi in self.made:
            assert (buf[:lo] == GUARD).all() and (buf[hi:] == GUARD).all(), what


def make(d, dt, N, G):
    rng = np.random.default_rng(d)
    t = dict(X=rows(rng, N, d, dt), Y=rows(rng, N, d, dt, 0.5), w_post=vec(rng, d, dt, 1.0), gate=vec(rng, (G, d), dt, 0.3),
             w_pre=vec(rng, d, dt, 1.0), gX_out=rows(rng, N, d, dt, 1e-3), gH=rows(rng, N, d, dt, 1e-3))
    kw = dict(res_scale=0.7, eps=1e-5, p=0.1, seed=3, offset=1)
    b = {k: n64(v) for k, v in t.items()}
    ab = {k: np.abs(v) for k, v in b.items()}
    edge = ("X", "Y", "w_post", "gate", "w_pre")
    xr, hr = stage.norm(*(b[k] for k in edge), **kw)
    size, _ = stage.norm(ab["X"], ab["Y"], ab["w_post"], ab["gate"], None, **kw)
    r = 1 / np.sqrt((xr ** 2).mean(1, keepdims=True) + 1e-5)
    hsize = ab["w_pre"] * r * size + np.abs(hr) * (1 + np.sqrt((size ** 2).mean(1, keepdims=True)) * r)
    x = torch.from_numpy(xr.astype(np.float32)).to(DT[dt]).to(DEV)
    args = (b["gX_out"], b["gH"], n64(x), b["Y"], b["w_post"], b["gate"], b["w_pre"])
    t["X_out"] = x
    return t, kw, (xr, size, hr, hsize), (stage.norm_bwd(*args, **kw), stage.norm_bwd(*args, **kw, size=True))


def run(t, kw, fwd, bwd, dt, N, d, G, shift_in, shift_out, what):
    f32 = torch.float32
    x, h = shift_out.empty((N, d), DT[dt]), shift_out.empty((N, d), DT[dt])
    lac.stage_norm(t["X"], t["Y"], t["w_post"], t["gate"], t["w_pre"], X_out=x, H=h, **kw)
    near(x, fwd[0], fwd[1], DT[dt], steps(d), f"X_out, {what}")
    near(h, fwd[2], fwd[3], DT[dt], steps(d), f"H, {what}")
    out = dict(gX=shift_out.empty((N, d), DT[dt]), gY=shift_out.empty((N, d), DT[dt]), g_w_post=shift_out.empty((d,), f32),
               g_gate=shift_out.empty((G, d), f32), g_w_pre=shift_out.empty((d,), f32))
    lac.stage_norm_bwd(t["gX_out"], t["gH"], t["X_out"], t["Y"], t["w_post"], t["gate"], t["w_pre"], **kw, **out)
    for k, v in out.items():
        sums = k not in ("gX", "gY")
        near(v, bwd[0][k], bwd[1][k], f32 if sums else DT[dt], 4 * steps(d) + (N if sums else 0), f"{k}, {what}")
    shift_in.check(what)
    shift_out.check(what)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", WIDTHS)
def test_edge_at_any_address(d, dt):
    N, G = 11, 1
    t, kw, fwd, bwd = make(d, dt, N, G)
    for by_in, by_out in ((1, 0), (0, 1), (1, 1), (3, 2)):
        si, so = Shifted(by_in), Shifted(by_out)
        s = {k: si.copy(v) for k, v in t.items()}
        run(s, kw, fwd, bwd, dt, N, d, G, si, so, f"inputs moved by {by_in}, outputs by {by_out}")


@pytest.mark.parametrize("d", [6, 64, 1000, 1003, 2050])
def test_edge_with_one_tensor_at_an_odd_address(d):
    # a weight at a 2-byte boundary beside aligned rows, and rows at one beside aligned weights
    N, G = 6, 3
    t, kw, fwd, bwd = make(d, "bf16", N, G)
    for name in t:
        si, so = Shifted(1), Shifted(0)
        run({**t, name: si.copy(t[name])}, kw, fwd, bwd, "bf16", N, d, G, si, so, f"{name} moved")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [7, 72, 131, 1003, 2050])
def test_edge_at_any_address_with_a_gate_per_token(d, dt):
    N = G = 1031
    t, kw, fwd, bwd = make(d, dt, N, G)
    for by_in, by_out in ((1, 0), (0, 1), (1, 1)):
        si, so = Shifted(by_in), Shifted(by_out)
        run({k: si.copy(v) for k, v in t.items()}, kw, fwd, bwd, dt, N, d, G, si, so,
            f"inputs moved by {by_in}, outputs by {by_out}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [5, 64, 1003, 1025, 2050, 8190])
def test_forms_without_a_block_or_a_norm_at_any_address(d, dt):
    # the plain residual and norm (X + Y, norm behind it), the norm alone, and their gradients
    N = 9
    rng = np.random.default_rng(d)
    si, so = Shifted(1), Shifted(1)
    X, Y, gx, gh = (si.copy(rows(rng, N, d, dt)) for _ in range(4))
    w = si.copy(vec(rng, d, dt, 1.0))
    x, h = so.empty((N, d), DT[dt]), so.empty((N, d), DT[dt])
    lac.stage_norm(X, Y, w_pre=w, X_out=x, H=h)
    xr, hr = stage.norm(n64(X), n64(Y), w_pre=n64(w))
    size = np.abs(n64(X)) + np.abs(n64(Y))
    r = 1 / np.sqrt((xr ** 2).mean(1, keepdims=True) + 1e-5)
    near(x, xr, size, DT[dt], steps(d), "X_out")
    near(h, hr, np.abs(n64(w)) * r * size + np.abs(hr) * (1 + np.sqrt((size ** 2).mean(1, keepdims=True)) * r), DT[dt],
         steps(d), "H")
    x2 = si.copy(X)  # in place
    lac.stage_norm(x2, Y, w_pre=w, X_out=x2)
    assert torch.equal(x2, x)
    y2 = si.copy(Y)
    lac.stage_norm(X, y2, w_pre=w, X_out=y2)
    assert torch.equal(y2, x)
    hn = so.empty((N, d), DT[dt])
    lac.stage_norm(x, w_pre=w, H=hn, store_x=False)
    near(hn, stage.norm(n64(x), w_pre=n64(w))[1], 2 * np.abs(stage.norm(n64(x), w_pre=n64(w))[1]), DT[dt], steps(d), "H alone")
    for g, y in ((gx, Y), (gx, None), (None, None)):
        args = (None if g is None else n64(g), n64(gh), n64(x), None if y is None else n64(y), None, None, n64(w), 1.0, 1e-5,
                0.0, 0, 0)
        ref, big = stage.norm_bwd(*args), stage.norm_bwd(*args, size=True)
        out = dict(gX=so.empty((N, d), DT[dt]), g_w_pre=so.empty((d,), torch.float32))
        if y is not None:
            out["gY"] = so.empty((N, d), DT[dt])
        lac.stage_norm_bwd(g, gh, x, y, w_pre=w, **out)
        for k, v in out.items():
            near(v, ref[k], big[k], torch.float32 if k == "g_w_pre" else DT[dt], 4 * steps(d) + N, k)
    si.check("inputs")
    so.check("outputs")
