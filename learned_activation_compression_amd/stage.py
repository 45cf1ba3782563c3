"""Binding of the pipeline-stage operators (include/mapl_stage.h): dropout from
a counter-based generator, the fused edge of a transformer block with its
backward pass, and matrix products in 8-bit floating point.

As in the rest of the package each function has the name of the C entry point
it wraps and marshals arguments only.  Outputs, packs and workspaces that are
not given are allocated on the stream that the call runs on, so with an
explicit `stream` the caller orders the inputs, and nothing else, against it.
"""
from __future__ import annotations

import ctypes
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


# the current stream's handle without a Stream object around it (3 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


class _On:
    """Runs a call on the device of its tensors, and allocates on its stream."""

    __slots__ = ("device", "index", "other", "stream", "side", "handle")

    def __init__(self, like: torch.Tensor, stream):
        _dev(like, "the first tensor")
        self.device = like.device
        self.index = index = self.device.index
        self.other = torch.cuda.device(index) if torch.cuda.current_device() != index else None
        self.stream = stream
        self.side = torch.cuda.stream(stream) if stream is not None else None

    def __enter__(self):
        if self.other is not None:
            self.other.__enter__()
        if self.side is not None:
            self.side.__enter__()
        self.handle = _raw_stream(self.index) if self.stream is None else self.stream.cuda_stream
        return self

    def __exit__(self, *exc):
        if self.side is not None:
            self.side.__exit__(*exc)
        if self.other is not None:
            self.other.__exit__(*exc)

    def ptr(self, t, name, dtype=None, shape=None):
        """Device pointer of an optional tensor of this call's device."""
        if t is None:
            return None
        try:
            if t.get_device() == self.index and t.is_contiguous() and (dtype is None or t.dtype is dtype) and \
                    (shape is None or t.shape == shape):
                return t.data_ptr()
        except AttributeError:
            pass
        p = _dev(t, name, dtype)  # names what is wrong
        if t.device != self.device:
            raise MaplError(-1, "binding", f"{name} is on {t.device}, not {self.device}")
        if shape is not None and t.shape != shape:
            raise MaplError(-2, "binding", f"{name} must be {list(shape)}, got {list(t.shape)}")
        return p

    def empty(self, shape, dtype):
        return torch.empty(shape, dtype=dtype, device=self.device)

    def bytes(self, buf, need, name):
        """A caller's byte buffer or a new one: (tensor, pointer, size)."""
        if buf is None:
            if need == 0:
                return None, None, 0
            buf = self.empty(need, torch.uint8)
            return buf, buf.data_ptr(), need
        return buf, self.ptr(buf, name), buf.numel() * buf.element_size()


def _rows(t: torch.Tensor, name: str):
    if t.dim() < 2:
        raise MaplError(-2, "binding", f"{name} must be [..., N, d]")
    d = t.shape[-1]
    n = 1
    for s in t.shape[:-1]:
        n *= s
    return n, d


def _u(v, name) -> int:
    if not 0 <= int(v) < 1 << 64:
        raise MaplError(-4, "binding", f"{name} must be in [0, 2^64)")
    return int(v)


def stage_dropout(X, p, seed, offset=0, Y=None, stream=None) -> torch.Tensor:
    """Y = keep ? X / (1 - p) : 0, the mask a function of (seed, offset + row,
    column).  The gradient is the same call on dL/dY; Y may be X."""
    N, d = _rows(X, "X")
    with _On(X, stream) as on:
        if Y is None:
            Y = torch.empty_like(X)
        _check(_stage_lib().stage_dropout(on.ptr(X, "X"), on.ptr(Y, "Y", X.dtype, X.shape), float(p),
                                          _u(seed, "seed"), _u(offset, "offset"), N, d, _dt(X), on.handle),
               "stage_dropout")
    return Y


def stage_norm(X, Y=None, w_post=None, gate=None, w_pre=None, res_scale=1.0, eps=1e-5, p=0.0, seed=0, offset=0,
               X_out=None, H=None, store_x=True, stream=None):
    """X_out = res_scale X + gate * (w_post * rmsnorm(dropout(Y))) and
    H = w_pre * rmsnorm(X_out).  Returns (X_out, H); H is None without w_pre,
    X_out is None with store_x = False.  X, Y [..., N, d]; gate [G, d] with G
    dividing the number of rows."""
    N, d = _rows(X, "X")
    dt = X.dtype
    with _On(X, stream) as on:
        if X_out is None and store_x:
            X_out = torch.empty_like(X)
        if H is None and w_pre is not None:
            H = torch.empty_like(X)
        G = 0 if gate is None else gate.shape[0]
        _check(_stage_lib().stage_norm(on.ptr(X, "X"), on.ptr(Y, "Y", dt, X.shape), on.ptr(w_post, "w_post", dt, (d,)),
                                       on.ptr(gate, "gate", dt, (G, d)), on.ptr(w_pre, "w_pre", dt, (d,)),
                                       on.ptr(X_out, "X_out", dt, X.shape), on.ptr(H, "H", dt, X.shape),
                                       float(res_scale), float(eps), float(p), _u(seed, "seed"),
                                       _u(offset, "offset"), N, d, G, _dt(X), on.handle), "stage_norm")
    return X_out, H


def stage_norm_bwd_workspace_bytes(N: int, d: int, gate_rows: int = 0) -> int:
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
    N, d = _rows(like, "gX_out")
    dt, shape = like.dtype, like.shape
    with _On(like, stream) as on:
        G = 0 if gate is None else gate.shape[0]

        def grad(buf, want, size):
            if buf is not None or not want:
                return buf if want else None
            return torch.zeros(size, dtype=torch.float32, device=on.device) if accumulate else \
                on.empty(size, torch.float32)

        gX = torch.empty_like(like) if gX is None else gX
        gY = None if Y is None else torch.empty_like(like) if gY is None else gY
        g_w_post = grad(g_w_post, w_post is not None, (d,))
        g_gate = grad(g_gate, gate is not None, (G, d))
        g_w_pre = grad(g_w_pre, gH is not None, (d,))
        lib = _stage_lib()
        need = 0 if w_post is None and gate is None and gH is None else \
            int(lib.stage_norm_bwd_workspace_bytes(N, d, G))
        ws, ws_ptr, ws_size = on.bytes(ws, need, "ws")
        _check(lib.stage_norm_bwd(
            on.ptr(gX_out, "gX_out", dt, shape), on.ptr(gH, "gH", dt, shape), on.ptr(X_out, "X_out", dt, shape),
            on.ptr(Y, "Y", dt, shape), on.ptr(w_post, "w_post", dt, (d,)), on.ptr(gate, "gate", dt, (G, d)),
            on.ptr(w_pre, "w_pre", dt, (d,)), on.ptr(gX, "gX", dt, shape), on.ptr(gY, "gY", dt, shape),
            on.ptr(g_w_post, "g_w_post", torch.float32, (d,)), on.ptr(g_gate, "g_gate", torch.float32, (G, d)),
            on.ptr(g_w_pre, "g_w_pre", torch.float32, (d,)), int(bool(accumulate)), float(res_scale), float(eps),
            float(p), _u(seed, "seed"), _u(offset, "offset"), N, d, G, _dt(like), ws_ptr, ws_size, on.handle),
            "stage_norm_bwd")
    return gX, gY, g_w_post, g_gate, g_w_pre


# ------------------------------------------------------------------ 8 bits --

def fp8_pack_bytes(rows: int, cols: int) -> int:
    return int(_stage_lib().fp8_pack_bytes(rows, cols))


def fp8_pack(X, rows=True, cols=False, square=False, pk=None, pkT=None, stream=None):
    """X [..., R, C] to e4m3 with a scale per block of 128: pk is the operand
    [R][C] (rows = True), pkT that of the transpose (cols = True).  square
    scales 128 x 128 blocks (weights).  Returns (pk, pkT)."""
    R, C = _rows(X, "X")
    with _On(X, stream) as on:
        pk, pk_ptr, pk_size = on.bytes(pk, fp8_pack_bytes(R, C), "pk") if rows else (None, None, 0)
        pkT, pkT_ptr, pkT_size = on.bytes(pkT, fp8_pack_bytes(C, R), "pkT") if cols else (None, None, 0)
        _check(_stage_lib().fp8_pack(on.ptr(X, "X"), pk_ptr, pk_size, pkT_ptr, pkT_size, int(bool(square)), R, C,
                                     _dt(X), on.handle), "fp8_pack")
    return pk, pkT


def fp8_unpack(pk, rows: int, cols: int, dtype=torch.float32, X=None, stream=None) -> torch.Tensor:
    """The values [rows][cols] that a pack stands for."""
    with _On(pk, stream) as on:
        if X is None:
            X = on.empty((rows, cols), dtype)
        _check(_stage_lib().fp8_unpack(on.ptr(pk, "pk"), pk.numel() * pk.element_size(),
                                       on.ptr(X, "X", None, (rows, cols)), rows, cols, _dt(X), on.handle),
               "fp8_unpack")
    return X


def fp8_gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(_stage_lib().fp8_gemm_workspace_bytes(M, N, K))


def fp8_gemm(pkA, pkB, M: int, N: int, K: int, dtype=torch.bfloat16, C=None, accumulate=False, ws=None,
             stream=None) -> torch.Tensor:
    """C [M][N] (+)= A B^T for packs of A [M][K] and B [N][K]; accumulate adds
    into a given fp32 C."""
    with _On(pkA, stream) as on:
        if C is None:
            if accumulate:
                raise MaplError(-1, "fp8_gemm", "accumulate needs C")
            C = on.empty((M, N), dtype)
        lib = _stage_lib()
        ws, ws_ptr, ws_size = on.bytes(ws, int(lib.fp8_gemm_workspace_bytes(M, N, K)), "ws")
        _check(lib.fp8_gemm(on.ptr(pkA, "pkA"), pkA.numel() * pkA.element_size(), on.ptr(pkB, "pkB"),
                            pkB.numel() * pkB.element_size(), on.ptr(C, "C", None, (M, N)), int(bool(accumulate)), M,
                            N, K, _dt(C), ws_ptr, ws_size, on.handle), "fp8_gemm")
    return C
