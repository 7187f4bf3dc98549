"""Plain numpy forms of the routed-expert operators, in binary64 and by loops
over tokens, picks and groups: what the tests compare the kernels with."""
import numpy as np

U = 2.0 ** -24           # half a unit in the last place of fp32


def rows_needed(T, E, k, align):
    picks = T * k
    return -(-(picks + min(E, picks) * (align - 1)) // align) * align


def route(z, valid, k, normalize, align, M):
    """z: float64 [T, E] (the logits' exact values)."""
    T, E = z.shape
    idx = np.full((T, k), -1, np.int32)
    weight = np.zeros((T, k))
    p = np.zeros((T, E))
    live = 0
    groups = [[] for _ in range(E)]
    for t in range(T):
        if valid is not None and not valid[t]:
            continue
        row = z[t]
        if np.isnan(row).any() or (row == np.inf).any():
            live += 1
            p[t] = np.nan
            weight[t] = np.nan
            continue
        if not (row > -np.inf).any():
            continue
        live += 1
        e = np.exp(row - row.max())
        p[t] = e / e.sum()
        picks = [int(i) for i in np.lexsort((np.arange(E), -row))[:k] if row[i] > -np.inf]
        w = p[t][picks]
        if normalize:
            w = np.exp(row[picks] - row.max())
            w = w / w.sum()
        for j, e_ in enumerate(picks):
            idx[t, j] = e_
            weight[t, j] = w[j]
            groups[e_].append((t, j))
    counts = np.array([len(g) for g in groups], np.int32)
    slot = np.full((T, k), -1, np.int32)
    src = np.full(M, -1, np.int32)
    offs = np.zeros(E, np.int32)
    at = 0
    for e in range(E):
        for r, (t, j) in enumerate(groups[e]):
            slot[t, j] = at + r
            src[at + r] = t * k + j
        at += -(-len(groups[e]) // align) * align
        offs[e] = at
    n = max(live, 1)
    prob = p.sum(0) / n
    loss = E * float((counts / (k * n) * prob).sum())
    return dict(idx=idx, weight=weight, slot=slot, src=src, counts=counts, offs=offs, live=live, prob=prob, loss=loss,
                p=p)


def route_spread(z):
    """The largest distance of a finite score from its row's largest."""
    with np.errstate(invalid="ignore"):
        d = np.where(np.isfinite(z), z.max(1, keepdims=True) - z, 0.0)
    return float(np.nanmax(np.where(np.isfinite(d), d, 0.0))) if d.size else 0.0


def route_grad(z, r, k, normalize, dweight, dloss):
    """(dlogits, the magnitudes that went into each of them)."""
    T, E = z.shape
    n = max(r["live"], 1)
    base = dloss * E * r["counts"].astype(np.float64) / (k * n) / n
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        p = r["p"][t]
        if np.isnan(p).any():
            out[t] = np.nan
            continue
        if p.sum() == 0:
            continue
        a, up, v = base.copy(), np.zeros(E), np.zeros(E)
        for j in range(k):
            if r["idx"][t, j] >= 0:
                up[r["idx"][t, j]] = dweight[t, j]
                v[r["idx"][t, j]] = r["weight"][t, j]
        if normalize:
            out[t] = v * (up - (v * up).sum())
            mag[t] = v * (np.abs(up) + (v * np.abs(up)).sum())
        else:
            a = a + up
        out[t] += p * (a - (p * a).sum())
        mag[t] += p * (np.abs(a) + (p * np.abs(a)).sum())
    return out, mag


def quantize(x):
    """x: float32 [T, K]; every operation in fp32, as the definition says."""
    T, K = x.shape
    floor = np.float32(127) * np.float32(2.0 ** -126)
    q = np.zeros((T, K), np.int8)
    s = np.empty(T, np.float32)
    for t in range(T):
        if not np.isfinite(x[t]).all():
            s[t] = np.nan
            continue
        a = np.float32(max(np.abs(x[t]).max() if K else np.float32(0), floor))
        q[t] = np.rint(x[t] * np.float32(np.float32(127) * np.float32(np.float32(1) / a))).astype(np.int8)
        s[t] = np.float32(a / np.float32(127))
    return q, s


def product(qa, sa, qb, sb, bias=None):
    """(C, the magnitudes that went into it) in binary64; sums in integers."""
    acc = (qa.astype(np.float64) @ qb.astype(np.float64).T)          # exact: below 2^53
    c = acc * sa.astype(np.float64)[:, None] * sb.astype(np.float64)[None]
    mag = np.abs(c)
    if bias is not None:
        c = c + bias.astype(np.float64)
        mag = mag + np.abs(bias.astype(np.float64))
    return c, mag


def group_ranges(offs, M):
    """The clamped, ascending row ranges that any offsets delimit."""
    out, at = [], 0
    for o in offs:
        end = max(at, min(max(int(o), 0), M))
        out.append((at, end))
        at = end
    return out


def combine(rows, slot, weight):
    T, k = slot.shape
    y, mag = np.zeros((T, rows.shape[1])), np.zeros((T, rows.shape[1]))
    for t in range(T):
        for j in range(k):
            if 0 <= slot[t, j] < rows.shape[0]:
                w = 1.0 if weight is None else float(weight[t, j])
                y[t] += w * rows[slot[t, j]]
                mag[t] += abs(w) * np.abs(rows[slot[t, j]])
    return y, mag
