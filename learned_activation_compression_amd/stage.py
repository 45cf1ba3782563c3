"""Binding of the pipeline-stage operators (include/mapl_stage.h): dropout from
a counter-based generator, the fused edge of a transformer block with its
backward pass, and matrix products in 8-bit floating point.

As in the rest of the package each function has the name of the C entry point
it wraps and marshals arguments only.  Outputs, packs and workspaces that are
not given are allocated on the stream that the call runs on, so with an
explicit `stream` the caller orders the inputs, and nothing else, against it.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import re

import torch

from . import (HEADER_PATH, MaplError, _check, _dev, _dt, _f32, _i32, _i64, _sz, _vp)
from . import load as _load

__all__ = [
    "stage_dropout", "stage_norm", "stage_norm_bwd_workspace_bytes", "stage_norm_bwd",
    "fp8_pack_bytes", "fp8_pack", "fp8_unpack", "fp8_gemm_workspace_bytes", "fp8_gemm",
]

STAGE_HEADER_PATH = os.path.join(os.path.dirname(HEADER_PATH), "mapl_stage.h")

_f64, _u64 = ctypes.c_double, ctypes.c_uint64
_STAGE_SIGS = {
    "stage_dropout": (_i32, [_vp, _vp, _f64, _u64, _u64, _i64, _i64, _i32, _vp]),
    "stage_norm": (_i32, [_vp] * 7 + [_f32, _f32, _f64, _u64, _u64, _i64, _i64, _i64, _i32, _vp]),
    "stage_norm_bwd_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "stage_norm_bwd": (_i32, [_vp] * 12 + [_i32, _f32, _f32, _f64, _u64, _u64, _i64, _i64, _i64, _i32, _vp, _sz, _vp]),
    "fp8_pack_bytes": (_sz, [_i64, _i64]),
    "fp8_pack": (_i32, [_vp, _vp, _sz, _vp, _sz, _i32, _i64, _i64, _i32, _vp]),
    "fp8_unpack": (_i32, [_vp, _sz, _vp, _i64, _i64, _i32, _vp]),
    "fp8_gemm_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "fp8_gemm": (_i32, [_vp, _sz, _vp, _sz, _vp, _i32, _i64, _i64, _i64, _i32, _vp, _sz, _vp]),
}

_lib = None


def _stage_lib():
    global _lib
    if _lib is None:
        lib = _load()
        for name, (res, args) in _STAGE_SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def stage_symbols() -> list:
    """Names of the functions declared in include/mapl_stage.h."""
    with open(STAGE_HEADER_PATH) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    return re.findall(r"^\s*(?:int|size_t)\s+([a-z][a-z0-9_]*)\s*\(", text, flags=re.M)


# the current device and its current stream's handle without the objects around
# them, which cost more than the rest of a call's marshalling
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _elsewhere(like, name, stream) -> bool:
    """Whether a call has to enter the device of its first tensor or a stream first."""
    if stream is not None:
        _dev(like, name)
        return True
    try:
        index = like.get_device()
    except AttributeError:
        index = -1
    if index < 0:
        _dev(like, name)  # names what is wrong
    return index != _device()


@contextlib.contextmanager
def _there(like, stream):
    if stream is not None and stream.device != like.device:
        raise MaplError(-1, "binding", f"the stream is on {stream.device}, the tensors on {like.device}")
    with torch.cuda.device(like.device):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


def _ptr(t, name, index, dtype=None, shape=None):
    """Device pointer of an optional tensor on device `index`."""
    if t is None:
        return None
    try:
        if t.get_device() == index and t.is_contiguous() and (dtype is None or t.dtype is dtype) and \
                (shape is None or t.shape == shape):
            return t.data_ptr()
    except AttributeError:
        pass
    _dev(t, name, dtype)  # names what is wrong
    if t.get_device() != index:
        raise MaplError(-1, "binding", f"{name} is on {t.device}, not cuda:{index}")
    raise MaplError(-2, "binding", f"{name} must be {list(shape)}, got {list(t.shape)}")


def _bytes(buf, need, name, like):
    """A caller's byte buffer or a new one: (tensor, pointer, size)."""
    if buf is None:
        if need == 0:
            return None, None, 0
        buf = torch.empty(need, dtype=torch.uint8, device=like.device)
        return buf, buf.data_ptr(), need
    return buf, _ptr(buf, name, like.get_device()), buf.numel() * buf.element_size()


def _rows(t: torch.Tensor, name: str):
    shape = t.shape
    if len(shape) == 2:
        return shape
    if len(shape) < 2:
        raise MaplError(-2, "binding", f"{name} must be [..., N, d]")
    n = 1
    for s in shape[:-1]:
        n *= s
    return n, shape[-1]


def _u(v, name) -> int:
    if not 0 <= int(v) < 1 << 64:
        raise MaplError(-4, "binding", f"{name} must be in [0, 2^64)")
    return int(v)


def stage_dropout(X, p, seed, offset=0, Y=None, stream=None) -> torch.Tensor:
    """Y = keep ? X / (1 - p) : 0, the mask a function of (seed, offset + row,
    column).  The gradient is the same call on dL/dY; Y may be X."""
    if _elsewhere(X, "X", stream):
        with _there(X, stream):
            return stage_dropout(X, p, seed, offset, Y)
    N, d = _rows(X, "X")
    dev = X.get_device()
    if Y is None:
        Y = torch.empty_like(X)
    _check(_stage_lib().stage_dropout(_ptr(X, "X", dev), _ptr(Y, "Y", dev, X.dtype, X.shape), float(p),
                                      _u(seed, "seed"), _u(offset, "offset"), N, d, _dt(X), _raw_stream(dev)),
           "stage_dropout")
    return Y


def stage_norm(X, Y=None, w_post=None, gate=None, w_pre=None, res_scale=1.0, eps=1e-5, p=0.0, seed=0, offset=0,
               X_out=None, H=None, store_x=True, stream=None):
    """X_out = res_scale X + gate * (w_post * rmsnorm(dropout(Y))) and
    H = w_pre * rmsnorm(X_out).  Returns (X_out, H); H is None without w_pre,
    X_out is None with store_x = False.  X, Y [..., N, d]; gate [G, d] with G
    dividing the number of rows."""
    if _elsewhere(X, "X", stream):
        with _there(X, stream):
            return stage_norm(X, Y, w_post, gate, w_pre, res_scale, eps, p, seed, offset, X_out, H, store_x)
    N, d = _rows(X, "X")
    dt, shape, dev = X.dtype, X.shape, X.get_device()
    if X_out is None and store_x:
        X_out = torch.empty_like(X)
    if H is None and w_pre is not None:
        H = torch.empty_like(X)
    G = 0 if gate is None else gate.shape[0]
    _check(_stage_lib().stage_norm(
        _ptr(X, "X", dev), _ptr(Y, "Y", dev, dt, shape), _ptr(w_post, "w_post", dev, dt, (d,)),
        _ptr(gate, "gate", dev, dt, (G, d)), _ptr(w_pre, "w_pre", dev, dt, (d,)),
        _ptr(X_out, "X_out", dev, dt, shape), _ptr(H, "H", dev, dt, shape), float(res_scale), float(eps), float(p),
        _u(seed, "seed"), _u(offset, "offset"), N, d, G, _dt(X), _raw_stream(dev)), "stage_norm")
    return X_out, H


@functools.lru_cache(maxsize=4096)
def stage_norm_bwd_workspace_bytes(N: int, d: int, gate_rows: int = 0) -> int:
    """Workspace of stage_norm_bwd for these sizes."""
    return int(_stage_lib().stage_norm_bwd_workspace_bytes(N, d, gate_rows))


def stage_norm_bwd(gX_out=None, gH=None, X_out=None, Y=None, w_post=None, gate=None, w_pre=None, res_scale=1.0,
                   eps=1e-5, p=0.0, seed=0, offset=0, gX=None, gY=None, g_w_post=None, g_gate=None, g_w_pre=None,
                   accumulate=False, ws=None, stream=None):
    """Backward of stage_norm from the stored X_out (needed with gH) and Y.
    Returns (gX, gY, g_w_post, g_gate, g_w_pre), None where the input is absent;
    the last three are fp32, and accumulate adds into the given ones."""
    like = gX_out if gX_out is not None else gH
    if like is None:
        raise MaplError(-1, "stage_norm_bwd", "gX_out and gH are both None")
    if _elsewhere(like, "gX_out", stream):
        with _there(like, stream):
            return stage_norm_bwd(gX_out, gH, X_out, Y, w_post, gate, w_pre, res_scale, eps, p, seed, offset, gX, gY,
                                  g_w_post, g_gate, g_w_pre, accumulate, ws)
    N, d = _rows(like, "gX_out")
    dt, shape, dev, f32 = like.dtype, like.shape, like.get_device(), torch.float32
    G = 0 if gate is None else gate.shape[0]
    new = torch.zeros if accumulate else torch.empty
    if gX is None:
        gX = torch.empty_like(like)
    if Y is None:
        gY = None
    elif gY is None:
        gY = torch.empty_like(like)
    if w_post is None:
        g_w_post = None
    elif g_w_post is None:
        g_w_post = new(d, dtype=f32, device=like.device)
    if gate is None:
        g_gate = None
    elif g_gate is None:
        g_gate = new((G, d), dtype=f32, device=like.device)
    if gH is None:
        g_w_pre = None
    elif g_w_pre is None:
        g_w_pre = new(d, dtype=f32, device=like.device)
    need = 0 if w_post is None and gate is None and gH is None else stage_norm_bwd_workspace_bytes(N, d, G)
    ws, ws_ptr, ws_size = _bytes(ws, need, "ws", like)
    _check(_stage_lib().stage_norm_bwd(
        _ptr(gX_out, "gX_out", dev), _ptr(gH, "gH", dev, dt, shape), _ptr(X_out, "X_out", dev, dt, shape),
        _ptr(Y, "Y", dev, dt, shape), _ptr(w_post, "w_post", dev, dt, (d,)), _ptr(gate, "gate", dev, dt, (G, d)),
        _ptr(w_pre, "w_pre", dev, dt, (d,)), _ptr(gX, "gX", dev, dt, shape), _ptr(gY, "gY", dev, dt, shape),
        _ptr(g_w_post, "g_w_post", dev, f32, (d,)), _ptr(g_gate, "g_gate", dev, f32, (G, d)),
        _ptr(g_w_pre, "g_w_pre", dev, f32, (d,)), 1 if accumulate else 0, float(res_scale), float(eps), float(p),
        _u(seed, "seed"), _u(offset, "offset"), N, d, G, _dt(like), ws_ptr, ws_size, _raw_stream(dev)),
        "stage_norm_bwd")
    return gX, gY, g_w_post, g_gate, g_w_pre


# ------------------------------------------------------------------ 8 bits --

@functools.lru_cache(maxsize=4096)
def fp8_pack_bytes(rows: int, cols: int) -> int:
    """Bytes of the pack of an operand [rows][cols]."""
    return int(_stage_lib().fp8_pack_bytes(rows, cols))


def fp8_pack(X, rows=True, cols=False, square=False, pk=None, pkT=None, stream=None):
    """X [..., R, C] to e4m3 with a scale per block of 128: pk is the operand
    [R][C] (rows = True), pkT that of the transpose (cols = True).  square
    scales 128 x 128 blocks (weights).  Returns (pk, pkT)."""
    if _elsewhere(X, "X", stream):
        with _there(X, stream):
            return fp8_pack(X, rows, cols, square, pk, pkT)
    R, C = _rows(X, "X")
    pk, pk_ptr, pk_size = _bytes(pk, fp8_pack_bytes(R, C), "pk", X) if rows else (None, None, 0)
    pkT, pkT_ptr, pkT_size = _bytes(pkT, fp8_pack_bytes(C, R), "pkT", X) if cols else (None, None, 0)
    dev = X.get_device()
    _check(_stage_lib().fp8_pack(_ptr(X, "X", dev), pk_ptr, pk_size, pkT_ptr, pkT_size, 1 if square else 0, R, C,
                                 _dt(X), _raw_stream(dev)), "fp8_pack")
    return pk, pkT


def fp8_unpack(pk, rows: int, cols: int, dtype=torch.float32, X=None, stream=None) -> torch.Tensor:
    """The values [rows][cols] that a pack stands for."""
    if _elsewhere(pk, "pk", stream):
        with _there(pk, stream):
            return fp8_unpack(pk, rows, cols, dtype, X)
    if X is None:
        X = torch.empty((rows, cols), dtype=dtype, device=pk.device)
    dev = pk.get_device()
    _check(_stage_lib().fp8_unpack(_ptr(pk, "pk", dev), pk.numel() * pk.element_size(),
                                   _ptr(X, "X", dev, None, (rows, cols)), rows, cols, _dt(X), _raw_stream(dev)),
           "fp8_unpack")
    return X


@functools.lru_cache(maxsize=4096)
def fp8_gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    """Workspace of fp8_gemm for these sizes (0 where K is not split)."""
    return int(_stage_lib().fp8_gemm_workspace_bytes(M, N, K))


def fp8_gemm(pkA, pkB, M: int, N: int, K: int, dtype=torch.bfloat16, C=None, accumulate=False, ws=None,
             stream=None) -> torch.Tensor:
    """C [M][N] (+)= A B^T for packs of A [M][K] and B [N][K]; accumulate adds
    into a given fp32 C."""
    if _elsewhere(pkA, "pkA", stream):
        with _there(pkA, stream):
            return fp8_gemm(pkA, pkB, M, N, K, dtype, C, accumulate, ws)
    if C is None:
        if accumulate:
            raise MaplError(-1, "fp8_gemm", "accumulate needs C")
        C = torch.empty((M, N), dtype=dtype, device=pkA.device)
    ws, ws_ptr, ws_size = _bytes(ws, fp8_gemm_workspace_bytes(M, N, K), "ws", pkA)
    dev = pkA.get_device()
    _check(_stage_lib().fp8_gemm(_ptr(pkA, "pkA", dev), pkA.numel() * pkA.element_size(), _ptr(pkB, "pkB", dev),
                                 pkB.numel() * pkB.element_size(), _ptr(C, "C", dev, None, (M, N)),
                                 1 if accumulate else 0, M, N, K, _dt(C), ws_ptr, ws_size, _raw_stream(dev)),
           "fp8_gemm")
    return C
