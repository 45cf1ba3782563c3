"""Operators between a stage's boundary and its loss, in float64: causal
attention over packed sequences with its backward pass.  Plain definitions,
row by row.  `size = True` adds to each result the sum of its terms' absolute
values: the size against which an error of rounding in that sum is measured."""
import numpy as np


def starts(cu, N):
    """start[i] of each row's sequence, -1 for a row of none."""
    out = np.full(N, -1)
    for a, b in zip(cu[:-1], cu[1:]):
        out[a:b] = a
    return out


def attn(q, k, v, cu, scale):
    """q [N][Hq][D], k and v [N][Hkv][D] -> o, lse [Hq][N], sizes of o and of the
    scores [N][Hq] (the largest sum of absolute products a row sees).  Rows of no
    sequence are NaN."""
    N, Hq, D = q.shape
    G = Hq // k.shape[1]
    st = starts(cu, N)
    o, size = np.full((N, Hq, D), np.nan), np.full((N, Hq, D), np.nan)
    lse, ssize = np.full((Hq, N), np.nan), np.full((Hq, N), np.nan)
    for i in range(N):
        if st[i] < 0:
            continue
        r = slice(st[i], i + 1)
        for h in range(Hq):
            with np.errstate(invalid="ignore", over="ignore"):
                s = scale * (k[r, h // G] @ q[i, h])
                m = np.max(s)
                e = np.exp(s - m)
                l = np.sum(e)
                o[i, h] = (e / l) @ v[r, h // G]
                size[i, h] = (e / l) @ np.abs(v[r, h // G])
                lse[h, i] = m + np.log(l)
                ssize[h, i] = np.max(scale * (np.abs(k[r, h // G]) @ np.abs(q[i, h])))
    return o, lse, size, ssize


def attn_bwd(go, q, k, v, o, lse, cu, scale):
    """(gq, gk, gv) and their sizes, from the given o and lse."""
    N, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    st = starts(cu, N)
    g = {n: np.zeros(x.shape) for n, x in (("gq", q), ("gk", k), ("gv", v))}
    size = {n: np.zeros(x.shape) for n, x in (("gq", q), ("gk", k), ("gv", v))}
    for i in range(N):
        if st[i] < 0:
            continue
        r = slice(st[i], i + 1)
        for h in range(Hq):
            kh, vh = k[r, h // G], v[r, h // G]
            with np.errstate(invalid="ignore", over="ignore"):
                p = np.exp(scale * (kh @ q[i, h]) - lse[h, i])
                ds = scale * p * (vh @ go[i, h] - go[i, h] @ o[i, h])
                # each ds as the sum of its terms' absolute values
                dz = scale * p * (np.abs(vh) @ np.abs(go[i, h]) + np.abs(go[i, h]) @ np.abs(o[i, h]))
                g["gq"][i, h] = ds @ kh
                g["gk"][r, h // G] += ds[:, None] * q[i, h]
                g["gv"][r, h // G] += p[:, None] * go[i, h]
                size["gq"][i, h] = dz @ np.abs(kh)
                size["gk"][r, h // G] += dz[:, None] * np.abs(q[i, h])
                size["gv"][r, h // G] += p[:, None] * np.abs(go[i, h])
    for x in (*g.values(), *size.values()):
        x[st < 0] = np.nan
    return g, size
