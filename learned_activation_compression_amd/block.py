"""Binding of the operators between a stage's boundary and its loss
(include/mapl_block.h): the block edge with an 8-bit output, causal attention over
packed sequences and the distillation loss, the latter two with their backward
passes.

As in the rest of the package each function has the name of the C entry point
it wraps and marshals arguments only.  Outputs and workspaces that are not given
are allocated on the stream that the call runs on, so with an explicit `stream`
the caller orders the inputs, and nothing else, against it.
"""
from __future__ import annotations

import functools
import os
import re

import torch

from . import HEADER_PATH, MaplError, _check, _dt, _f32, _i32, _i64, _sz, _vp
from . import load as _load
from .stage import _bytes, _elsewhere, _f64, _ptr, _raw_stream, _rows, _there, _u, _u64, fp8_pack_bytes

__all__ = [
    "stage_norm_pack", "stage_attn", "stage_attn_bwd_workspace_bytes", "stage_attn_bwd",
    "stage_distill_workspace_bytes", "stage_distill", "stage_distill_bwd",
]

BLOCK_HEADER_PATH = os.path.join(os.path.dirname(HEADER_PATH), "mapl_block.h")

_BLOCK_SIGS = {
    "stage_norm_pack": (_i32, [_vp] * 8 + [_sz, _f32, _f32, _f64, _u64, _u64, _i64, _i64, _i64, _i32, _vp]),
    "stage_attn": (_i32, [_vp] * 6 + [_f32] + [_i64] * 9 + [_i32, _vp]),
    "stage_attn_bwd_workspace_bytes": (_sz, [_i64] * 4),
    "stage_attn_bwd": (_i32, [_vp] * 10 + [_f32] + [_i64] * 13 + [_i32, _vp, _sz, _vp]),
    "stage_distill_workspace_bytes": (_sz, [_i64, _i64]),
    "stage_distill": (_i32, [_vp] * 6 + [_f32] * 3 + [_i64] * 3 + [_i32, _vp, _sz, _vp]),
    "stage_distill_bwd": (_i32, [_vp] * 7 + [_f32] * 3 + [_i64] * 3 + [_i32, _vp]),
}

_lib = None


def _block_lib():
    global _lib
    if _lib is None:
        lib = _load()
        for name, (res, args) in _BLOCK_SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def block_symbols() -> list:
    """Names of the functions declared in include/mapl_block.h."""
    with open(BLOCK_HEADER_PATH) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    return re.findall(r"^\s*(?:int|size_t)\s+([a-z][a-z0-9_]*)\s*\(", text, flags=re.M)


# -------------------------------------------------------------- block edge --

def stage_norm_pack(X, Y=None, w_post=None, gate=None, w_pre=None, res_scale=1.0, eps=1e-5, p=0.0, seed=0, offset=0,
                    X_out=None, H=None, pkH=None, store_x=True, store_h=False, stream=None):
    """stage_norm whose H leaves as the 8-bit operand [N][d] of fp8_gemm, packed
    from H before its rounding.  Returns (X_out, H, pkH); X_out is None with
    store_x = False, H is None unless it is given or store_h = True."""
    if _elsewhere(X, "X", stream):
        with _there(X, stream):
            return stage_norm_pack(X, Y, w_post, gate, w_pre, res_scale, eps, p, seed, offset, X_out, H, pkH, store_x,
                                   store_h)
    N, d = _rows(X, "X")
    dt, shape, dev = X.dtype, X.shape, X.get_device()
    if X_out is None and store_x:
        X_out = torch.empty_like(X)
    if H is None and store_h:
        H = torch.empty_like(X)
    pkH, pk_ptr, pk_size = _bytes(pkH, fp8_pack_bytes(N, d), "pkH", X)
    G = 0 if gate is None else gate.shape[0]
    _check(_block_lib().stage_norm_pack(
        _ptr(X, "X", dev), _ptr(Y, "Y", dev, dt, shape), _ptr(w_post, "w_post", dev, dt, (d,)),
        _ptr(gate, "gate", dev, dt, (G, d)), _ptr(w_pre, "w_pre", dev, dt, (d,)),
        _ptr(X_out, "X_out", dev, dt, shape), _ptr(H, "H", dev, dt, shape), pk_ptr, pk_size, float(res_scale),
        float(eps), float(p), _u(seed, "seed"), _u(offset, "offset"), N, d, G, _dt(X), _raw_stream(dev)),
        "stage_norm_pack")
    return X_out, H, pkH


# --------------------------------------------------------------- attention --

def _heads(t, name, index, dtype, shape):
    """Pointer and leading dimension of rows of heads [N, H, D]: heads lie side by side, rows at any stride."""
    try:
        if t.shape == shape and t.dtype is dtype and t.get_device() == index:
            row, head, one = t.stride()
            N, H, D = shape
            # torch gives any stride to an axis of one
            if (one == 1 or D == 1) and (head == D or H == 1) and (row >= H * D or N <= 1):
                return t.data_ptr(), row if N > 1 else H * D
            raise MaplError(-2, "binding", f"{name}: heads must lie side by side and rows apart, strides are {t.stride()}")
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise MaplError(-1, "binding", f"{name} must be a device tensor")
    if t.get_device() != index:
        raise MaplError(-1, "binding", f"{name} is on {t.device}, not cuda:{index}")
    if t.dtype is not dtype:
        raise MaplError(-3, "binding", f"{name} must be {dtype}, got {t.dtype}")
    raise MaplError(-2, "binding", f"{name} must be {list(shape)}, got {list(t.shape)}")


def _attn_shape(Q, K):
    """The shapes of Q and its like, and of K and its like."""
    try:
        q, k = Q.shape, K.shape
    except AttributeError:
        raise MaplError(-1, "binding", "Q and K must be torch.Tensors") from None
    if len(q) != 3 or len(k) != 3:
        raise MaplError(-2, "binding", "Q and K must be [N, heads, D]")
    return q, (q[0], k[1], q[2])


def stage_attn(Q, K, V, cu, scale=None, O=None, lse=None, stream=None):
    """Causal attention over packed sequences.  Q [N, Hq, D], K and V
    [N, Hkv, D], rows at any stride (columns of a fused projection); cu [S + 1]
    int32, the sequences' edges; scale defaults to D ** -0.5.  Returns (O, lse):
    [N, Hq, D] and fp32 [Hq, N].  Rows outside the sequences are not written."""
    if _elsewhere(cu, "cu", stream):
        with _there(cu, stream):
            return stage_attn(Q, K, V, cu, scale, O, lse)
    qs, ks = _attn_shape(Q, K)
    N, Hq, D = qs
    dev, dt = cu.get_device(), Q.dtype
    q, ldq = _heads(Q, "Q", dev, dt, qs)
    k, ldk = _heads(K, "K", dev, dt, ks)
    v, ldv = _heads(V, "V", dev, dt, ks)
    if O is None:
        O = Q.new_empty(qs)
        o, ldo = O.data_ptr(), Hq * D
    else:
        o, ldo = _heads(O, "O", dev, dt, qs)
    if lse is None:
        lse = Q.new_empty((Hq, N), dtype=torch.float32)
    _check(_block_lib().stage_attn(
        q, k, v, _ptr(cu, "cu", dev, torch.int32), o, _ptr(lse, "lse", dev, torch.float32, (Hq, N)),
        D ** -0.5 if scale is None else scale, cu.numel() - 1, N, Hq, ks[1], D, ldq, ldk, ldv, ldo, _dt(Q),
        _raw_stream(dev)), "stage_attn")
    return O, lse


@functools.lru_cache(maxsize=4096)
def stage_attn_bwd_workspace_bytes(N: int, Hq: int, Hkv: int, D: int) -> int:
    """Workspace of stage_attn_bwd for these sizes."""
    return int(_block_lib().stage_attn_bwd_workspace_bytes(N, Hq, Hkv, D))


def stage_attn_bwd(gO, Q, K, V, O, lse, cu, scale=None, gQ=None, gK=None, gV=None, ws=None, stream=None):
    """Backward of stage_attn from its inputs, O and lse.  Returns (gQ, gK, gV);
    given ones may be columns of the fused projection's gradient."""
    if _elsewhere(cu, "cu", stream):
        with _there(cu, stream):
            return stage_attn_bwd(gO, Q, K, V, O, lse, cu, scale, gQ, gK, gV, ws)
    qs, ks = _attn_shape(Q, K)
    N, Hq, D = qs
    Hkv, dev, dt = ks[1], cu.get_device(), Q.dtype
    go, ldgo = _heads(gO, "gO", dev, dt, qs)
    q, ldq = _heads(Q, "Q", dev, dt, qs)
    k, ldk = _heads(K, "K", dev, dt, ks)
    v, ldv = _heads(V, "V", dev, dt, ks)
    o, ldo = _heads(O, "O", dev, dt, qs)
    gQ = Q.new_empty(qs) if gQ is None else gQ
    gK = Q.new_empty(ks) if gK is None else gK
    gV = Q.new_empty(ks) if gV is None else gV
    gq, ldgq = _heads(gQ, "gQ", dev, dt, qs)
    gk, ldgk = _heads(gK, "gK", dev, dt, ks)
    gv, ldgv = _heads(gV, "gV", dev, dt, ks)
    ws, ws_ptr, ws_size = _bytes(ws, stage_attn_bwd_workspace_bytes(N, Hq, Hkv, D), "ws", cu)
    _check(_block_lib().stage_attn_bwd(
        go, q, k, v, o, _ptr(lse, "lse", dev, torch.float32, (Hq, N)), _ptr(cu, "cu", dev, torch.int32), gq, gk, gv,
        D ** -0.5 if scale is None else scale, cu.numel() - 1, N, Hq, Hkv, D, ldgo, ldq, ldk, ldv, ldo, ldgq, ldgk,
        ldgv, _dt(Q), ws_ptr, ws_size, _raw_stream(dev)), "stage_attn_bwd")
    return gQ, gK, gV


# -------------------------------------------------------------------- loss --

@functools.lru_cache(maxsize=4096)
def stage_distill_workspace_bytes(N: int, V: int) -> int:
    """Workspace of stage_distill for these sizes (0 where rows are not split)."""
    return int(_block_lib().stage_distill_workspace_bytes(N, V))


def _teacher(Z, labels, t_ids, t_logits, N, dev):
    """Pointers of the labels and the teacher's entries, and K."""
    if (t_ids is None) != (t_logits is None):
        raise MaplError(-1, "binding", "t_ids and t_logits come together")
    K = 0 if t_ids is None else t_ids.shape[-1]
    lead = Z.shape[:-1]
    return (_ptr(labels, "labels", dev, torch.int32, lead), _ptr(t_ids, "t_ids", dev, torch.int32, (*lead, K)),
            _ptr(t_logits, "t_logits", dev, torch.float32, (*lead, K)), K)


def stage_distill(Z, labels=None, t_ids=None, t_logits=None, temperature=1.0, w_ce=1.0, w_kd=1.0, loss=None, stats=None,
                  ws=None, stream=None):
    """Loss of logits Z [..., V]: w_ce times the cross-entropy with labels [...]
    (int32, -1: none) plus w_kd times the divergence from the teacher's top logits
    t_logits [..., K] (fp32) at t_ids [..., K] (int32, -1: no entry), at the
    temperature.  Returns (loss [...], stats [..., 2]), fp32; stats is for
    stage_distill_bwd."""
    if _elsewhere(Z, "Z", stream):
        with _there(Z, stream):
            return stage_distill(Z, labels, t_ids, t_logits, temperature, w_ce, w_kd, loss, stats, ws)
    N, V = _rows(Z, "Z")
    dev, lead = Z.get_device(), Z.shape[:-1]
    if loss is None:
        loss = torch.empty(lead, dtype=torch.float32, device=Z.device)
    if stats is None:
        stats = torch.empty((*lead, 2), dtype=torch.float32, device=Z.device)
    y, ids, logits, K = _teacher(Z, labels, t_ids, t_logits, N, dev)
    ws, ws_ptr, ws_size = _bytes(ws, stage_distill_workspace_bytes(N, V), "ws", Z)
    _check(_block_lib().stage_distill(
        _ptr(Z, "Z", dev), y, ids, logits, _ptr(loss, "loss", dev, torch.float32, lead),
        _ptr(stats, "stats", dev, torch.float32, (*lead, 2)), float(temperature), float(w_ce), float(w_kd), N, V, K,
        _dt(Z), ws_ptr, ws_size, _raw_stream(dev)), "stage_distill")
    return loss, stats


def stage_distill_bwd(gloss, Z, stats, labels=None, t_ids=None, t_logits=None, temperature=1.0, w_ce=1.0, w_kd=1.0,
                      gZ=None, stream=None):
    """Gradient of stage_distill with respect to Z, given gloss [...] (fp32) and
    the forward call's stats and arguments.  gZ may be Z."""
    if _elsewhere(Z, "Z", stream):
        with _there(Z, stream):
            return stage_distill_bwd(gloss, Z, stats, labels, t_ids, t_logits, temperature, w_ce, w_kd, gZ)
    N, V = _rows(Z, "Z")
    dev, lead = Z.get_device(), Z.shape[:-1]
    if gZ is None:
        gZ = torch.empty_like(Z)
    y, ids, logits, K = _teacher(Z, labels, t_ids, t_logits, N, dev)
    _check(_block_lib().stage_distill_bwd(
        _ptr(gloss, "gloss", dev, torch.float32, lead), _ptr(Z, "Z", dev),
        _ptr(stats, "stats", dev, torch.float32, (*lead, 2)), y, ids, logits, _ptr(gZ, "gZ", dev, Z.dtype, Z.shape),
        float(temperature), float(w_ce), float(w_kd), N, V, K, _dt(Z), _raw_stream(dev)), "stage_distill_bwd")
    return gZ
