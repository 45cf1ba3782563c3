"""Operators between a stage's boundary and its loss, in float64: causal
attention over packed sequences and the distillation loss, with their backward
passes.  Plain definitions, row by row.  `size = True` adds to each result the sum of its terms' absolute
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


def _lse(x):
    m = np.max(x)
    if not np.isfinite(m):
        return m if m < 0 or not np.isnan(m) else np.nan
    return m + np.log(np.sum(np.exp(x - m)))


def _row(z, y, ids, t, T, w_ce, w_kd):
    """Label or None, the entries' ids and log-probabilities."""
    V = len(z)
    y = None if w_ce == 0 or y is None or not 0 <= y < V else y
    ok = np.zeros(0, dtype=bool) if w_kd == 0 else (ids >= 0) & (ids < V) & (t != -np.inf)
    ids, t = ids[:len(ok)][ok], t[:len(ok)][ok] / T
    return y, ids, t - _lse(t) if len(t) else t


def distill(Z, labels, t_ids, t_logits, T, w_ce, w_kd):
    """loss, stats and, row by row, the sum of the loss's terms in absolute value."""
    N = Z.shape[0]
    loss, stats, size = np.zeros(N), np.zeros((N, 2)), np.zeros(N)
    for n in range(N):
        z = Z[n]
        stats[n] = _lse(z), _lse(z / T)
        y, ids, logq = _row(z, None if labels is None else labels[n], t_ids[n], t_logits[n], T, w_ce, w_kd)
        if y is not None:
            loss[n] += w_ce * (stats[n, 0] - z[y])
            size[n] += abs(w_ce) * (abs(stats[n, 0]) + abs(z[y]))
        if len(ids):
            loss[n] += w_kd * np.sum(np.exp(logq) * (logq - (z[ids] / T - stats[n, 1])))
            size[n] += abs(w_kd) * np.sum(np.exp(logq) * (np.abs(logq) + np.abs(z[ids] / T) + abs(stats[n, 1])))
    return loss, stats, size


def distill_bwd(gloss, Z, labels, t_ids, t_logits, T, w_ce, w_kd):
    """gZ and the sum of each element's terms in absolute value."""
    g, size = np.zeros(Z.shape), np.zeros(Z.shape)
    for n in range(Z.shape[0]):
        z = Z[n]
        y, ids, logq = _row(z, None if labels is None else labels[n], t_ids[n], t_logits[n], T, w_ce, w_kd)
        for x, f in ((g, lambda v: v), (size, np.abs)):
            if y is not None:
                x[n] += f(gloss[n] * w_ce) * np.exp(z - _lse(z))
                x[n, y] += f(-gloss[n] * w_ce)
            if len(ids):
                x[n] += f(gloss[n] * w_kd / T) * np.exp(z / T - _lse(z / T))
                np.add.at(x[n], ids, f(-gloss[n] * w_kd / T) * np.exp(logq))
    return g, size
