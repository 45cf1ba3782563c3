"""Pipeline-stage operators in float64: dropout from Philox4x32-10, the edge of
a block (dropout, norms, gate, residual) with its backward pass, and rounding
to e4m3 with a power-of-two scale per block of 128.  Plain definitions."""
import numpy as np

M32 = np.uint64(0xFFFFFFFF)


# ----------------------------------------------------------------- dropout --

def philox4x32_10(ctr, key):
    """Philox4x32-10 (Salmon, Moraes, Dror, Shaw, SC 2011): ctr [..., 4] and key
    (k0, k1) as 32-bit words -> [..., 4] words (uint64 arrays holding 32 bits)."""
    c = [np.asarray(ctr[..., i], dtype=np.uint64) for i in range(4)]
    k0, k1 = int(key[0]), int(key[1])
    for _ in range(10):
        p0 = np.uint64(0xD2511F53) * c[0]
        p1 = np.uint64(0xCD9E8D57) * c[2]
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), p1 & M32,
             (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), p0 & M32]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, axis=-1)


def threshold(p: float) -> int:
    return int(np.floor(p * 65536 + 0.5))


def keep(N: int, d: int, p: float, seed: int, offset: int) -> np.ndarray:
    """bool [N, d]: the kept elements."""
    ctr = np.zeros((N, (d + 7) // 8, 4), dtype=np.uint64)
    row = (np.arange(N, dtype=object) + offset) % (1 << 64)
    ctr[..., 0] = np.arange((d + 7) // 8, dtype=np.uint64)[None, :]
    ctr[..., 1] = np.array([r & 0xFFFFFFFF for r in row], dtype=np.uint64)[:, None]
    ctr[..., 2] = np.array([r >> 32 for r in row], dtype=np.uint64)[:, None]
    w = philox4x32_10(ctr, (seed & 0xFFFFFFFF, seed >> 32))
    u = np.empty((N, w.shape[1], 8), dtype=np.int64)
    u[..., 0::2] = (w & np.uint64(0xFFFF)).astype(np.int64)
    u[..., 1::2] = (w >> np.uint64(16)).astype(np.int64)
    return u.reshape(N, -1)[:, :d] >= threshold(p)


def dropout(X, p, seed, offset):
    t = threshold(p)
    if t == 0:
        return np.array(X, dtype=np.float64)
    s = 65536.0 / (65536 - t) if t < 65536 else 0.0
    k = keep(X.shape[0], X.shape[1], p, seed, offset)
    out = np.zeros(X.shape)
    out[k] = X[k] * s
    return out


# -------------------------------------------------------------- block edge --

def _rms(x, eps):
    return 1.0 / np.sqrt(np.mean(x * x, axis=1, keepdims=True) + eps)


def _gate(gate, N):
    return 1.0 if gate is None else np.repeat(gate, N // gate.shape[0], axis=0)


def norm(X, Y=None, w_post=None, gate=None, w_pre=None, res_scale=1.0, eps=1e-5, p=0.0, seed=0, offset=0):
    """(X_out, H); H is None without w_pre."""
    x = res_scale * X
    if Y is not None:
        v = dropout(Y, p, seed, offset)
        if w_post is not None:
            v = w_post * v * _rms(v, eps)
        x = x + _gate(gate, X.shape[0]) * v
    return x, None if w_pre is None else w_pre * x * _rms(x, eps)


def norm_bwd(gX_out, gH, X_out, Y, w_post, gate, w_pre, res_scale, eps, p, seed, offset, size=False):
    """dict of the gradients.  size = True takes every term by its absolute
    value: the size against which an error of rounding in that sum is measured."""
    f = np.abs if size else (lambda v: v)
    sub = np.add if size else np.subtract
    like = gX_out if gX_out is not None else gH
    N, d = like.shape
    t = np.zeros((N, d)) if gX_out is None else f(gX_out)
    out = {}
    if gH is not None:
        r, a, x = _rms(X_out, eps), f(gH * w_pre), f(X_out)
        t = t + r * sub(a, x * r * r * np.mean(a * x, axis=1, keepdims=True))
        out["g_w_pre"] = np.sum(f(gH * X_out) * r, axis=0)
    out["gX"] = f(np.asarray(res_scale)) * t
    if Y is not None:
        u0 = dropout(Y, p, seed, offset)
        q = _rms(u0, eps) if w_post is not None else 1.0
        u, w, g = f(u0), 1.0 if w_post is None else f(w_post), f(_gate(gate, N))
        if gate is not None:
            out["g_gate"] = (t * w * q * u).reshape(gate.shape[0], -1, d).sum(axis=1)
        b = t * g * w
        if w_post is not None:
            out["g_w_post"] = np.sum(t * g * q * u, axis=0)
            b = q * sub(b, u * q * q * np.mean(b * u, axis=1, keepdims=True))
        out["gY"] = dropout(b, p, seed, offset)
    return out


# ------------------------------------------------------------------- 8 bits --

def _grid():
    """The finite magnitudes of OCP e4m3, in the order of their codes."""
    return np.array([m * 2.0 ** -9 for m in range(8)] +
                    [(1 + f / 8) * 2.0 ** (e - 7) for e in range(1, 16) for f in range(8)][:-1])


GRID = _grid()


def e4m3(x):
    """The nearest e4m3 value, ties to the even code; |x| <= 448."""
    a = np.abs(x)
    hi = np.clip(np.searchsorted(GRID, a, side="left"), 1, len(GRID) - 1)
    lo = hi - 1
    dl, dh = a - GRID[lo], GRID[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return np.copysign(GRID[code], x)


def round_blocks(X, square=False):
    """The values that a pack of X [R][C] (blocks along its columns) stands for."""
    R, C = X.shape
    b = 128 if square else 1
    out = np.empty((R, C))
    for r0 in range(0, R, b):
        for c0 in range(0, C, 128):
            x = X[r0:r0 + b, c0:c0 + 128]
            fin = np.isfinite(x)
            top = np.max(np.abs(x[fin]), initial=0.0)
            s = -126
            while top > 448.0 * 2.0 ** s:
                s += 1
            y = np.full(x.shape, np.nan)
            y[fin] = e4m3(x[fin] * 2.0 ** -s) * 2.0 ** s
            out[r0:r0 + b, c0:c0 + 128] = y
    return out


def cut_products(a, b):
    """a b^T where, of each 8 columns' products, those bits count that are at
    least 2^-13 of 2^e, e the largest sum of two factors' exponents among the 8."""
    def exponent(x):
        return np.where(x != 0, np.frexp(x)[1] - 1, -10000)

    def by_eights(x):
        return np.concatenate([x, np.zeros(x.shape[:1] + (-x.shape[1] % 8,))], axis=1).reshape(x.shape[0], -1, 8)

    a, b = by_eights(a)[:, None], by_eights(b)[None]
    e = np.max(exponent(a) + exponent(b), axis=3, keepdims=True)
    q = np.ldexp(1.0, np.maximum(e, -1000) - 13)
    return np.sum(np.trunc(a * b / q) * q, axis=(2, 3))
