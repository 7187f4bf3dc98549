"""Scored routing in binary64, by numpy, token by token: what the tests compare
the kernels with, and how far fp32 may be from it."""
import numpy as np

U = 2.0 ** -24
EPS = 1e-20
GONE = 2.0 ** -126       # e^x ends there


def scores(z, kind):
    """s of one row of finite or -inf logits."""
    with np.errstate(over="ignore"):
        if kind == "sigmoid":
            return 1 / (1 + np.exp(-z))
        e = np.exp(z - z.max())
        return e / e.sum()


def picks(z, s, bias, groups, top, best, k):
    """The picks of one row, in order."""
    E = len(z)
    can = z > -np.inf
    if bias is not None:
        can = can & np.isfinite(bias)
    u = s if bias is None else s + np.where(np.isfinite(bias), bias, 0.0)
    size = E // groups
    if top < groups:
        worth = []
        for g in range(groups):
            v = np.sort(u[g * size:(g + 1) * size][can[g * size:(g + 1) * size]])[::-1][:best]
            worth.append(v.sum() if len(v) else -np.inf)
        order = sorted(range(groups), key=lambda g: (-worth[g], g))[:top]
        stays = np.zeros(groups, bool)
        stays[order] = True
        can = can & np.repeat(stays, size)
    v = z if bias is None else u
    at = np.flatnonzero(can)
    return [int(e) for e in at[np.lexsort((at, -v[at]))][:k]]


def route(z, k, kind, bias=None, groups=1, top=1, best=2, normalize=True, scale=1.0, valid=None, align=1, M=0):
    """z: float64 [T, E] (the logits' exact values)."""
    T, E = z.shape
    idx, weight = np.full((T, k), -1, np.int32), np.zeros((T, k))
    s, share = np.zeros((T, E)), np.zeros((T, E))
    live, spread, members = 0, 0.0, [[] for _ in range(E)]
    for t in range(T):
        row = z[t]
        if valid is not None and not valid[t]:
            continue
        if np.isnan(row).any() or (row == np.inf).any():
            live += 1
            s[t] = share[t] = weight[t] = np.nan
            continue
        if not (row > -np.inf).any():
            continue
        live += 1
        s[t] = scores(row, kind)
        share[t] = s[t] / (s[t].sum() + EPS) if kind == "sigmoid" else s[t]
        fin = row[row > -np.inf]
        spread = max(spread, fin.max() - fin.min())
        p = picks(row, s[t], bias, groups, top, best, k)
        w = s[t][p]
        if normalize:
            w = w / (w.sum() + EPS)
        for j, e in enumerate(p):
            idx[t, j], weight[t, j] = e, scale * w[j]
            members[e].append((t, j))
    counts = np.array([len(m) for m in members], np.int32)
    slot, src, offs = np.full((T, k), -1, np.int32), np.full(M, -1, np.int32), np.zeros(E, np.int32)
    at = 0
    for e in range(E):
        for r, (t, j) in enumerate(members[e]):
            slot[t, j] = at + r
            src[at + r] = t * k + j
        at += -(-len(members[e]) // align) * align
        offs[e] = at
    n = max(live, 1)
    prob = share.sum(0) / n
    return dict(idx=idx, weight=weight, slot=slot, src=src, counts=counts, offs=offs, live=live, prob=prob,
                loss=E * float((counts / (k * n) * prob).sum()), s=s, spread=spread)


def weight_error(r, k, E, kind, normalize, scale):
    """A sigmoid score is within 16 u (and 2^-126); a softmax one within (6 D + 2
    E + 32) u for scores D apart, as mx_route's.  Sums of k, a division and the
    scale on top, and the scores' own errors twice where they are divided."""
    one = 16 * U if kind == "sigmoid" else (6 * r["spread"] + 2 * E + 32) * U
    w = np.abs(r["weight"])
    if not normalize:
        return w * (one + 4 * U) + GONE * abs(scale)
    s = np.where(r["idx"] >= 0, np.take_along_axis(r["s"], np.maximum(r["idx"], 0), 1), 0.0)
    return w * (2 * one + (k + 6) * U) + (k + 1) * GONE * abs(scale) / (s.sum(1, keepdims=True) + EPS)


def grad(z, r, k, kind, normalize, scale, dweight, dloss):
    """(dlogits, the magnitudes that went into each of them)."""
    T, E = z.shape
    n = max(r["live"], 1)
    a = dloss * E * r["counts"].astype(np.float64) / (k * n) / n
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        s = r["s"][t]
        if np.isnan(s).any():
            out[t] = np.nan
            continue
        if not (z[t] > -np.inf).any() or s.sum() == 0:
            continue
        p = r["idx"][t][r["idx"][t] >= 0]
        d = scale * dweight[t][:len(p)]
        total = s[p].sum() + EPS
        dm = np.abs(d)
        if normalize:
            w = s[p] / total
            dm = (np.abs(d) + (np.abs(d) * w).sum()) / total
            d = (d - (d * w).sum()) / total
        up, um = np.zeros(E), np.zeros(E)
        up[p], um[p] = d, dm
        if kind == "sigmoid":
            m = s.sum() + EPS
            up, um = up + (a - (a * s).sum() / m) / m, um + (np.abs(a) + (np.abs(a) * s).sum() / m) / m
            slope = s * (1 / (1 + np.exp(np.minimum(z[t], 700))))
            out[t], mag[t] = up * slope, um * slope
        else:
            out[t] = s * (a + up - (s * (a + up)).sum())
            mag[t] = s * (np.abs(a) + um + (s * (np.abs(a) + um)).sum())
    return out, mag
