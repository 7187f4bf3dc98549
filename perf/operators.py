"""What is measured of the routed-expert operators around the casts and contractions.

The operators, and the calls that run them:
  routing     mx_route, mx_route_grad: softmax scores, the k best experts of each token, counts per expert, the
              padded group ends and row map that the grouped casts and contractions take, and the balance loss
              with its gradient
  dispatch    mx_dispatch: token rows copied to their experts' rows
  product     i8_linear, mx_dispatch_i8 + i8_grouped_gemm_rows: matrix products in 8-bit integers with a scale for
              each token and each output channel, dense and by expert, with the activations quantized on the way
  combine     mx_combine, mx_combine_grad: the weighted sum of each token's expert rows, and its gradient

A token that is not valid (padding of a batch) may hold anything, NaN too.  A logit of -inf is an expert that the
token may not use.  Rows of the padded buffer that belong to no token are zero.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"


# ---------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one token of one sequence while it is being decoded
        dict(name="route_token", op="route", T=1, E=64, k=4, dtype="bf16", align=1, train=False, normalize=True),
        # a training step's tokens on one GPU, 64 experts as in the grouped cast's workload
        dict(name="route_train", op="route", T=16384, E=64, k=8, dtype="bf16", align=128, train=True, normalize=True),
        # a long-sequence batch over many experts, scores kept in fp32 and weights not renormalized
        dict(name="route_large", op="route", T=131072, E=256, k=8, dtype="f32", align=128, train=True, normalize=False),
        # a small ragged batch of fp32 rows
        dict(name="dispatch_odd", op="dispatch", T=37, N=1111, E=10, k=3, dtype="f32", align=1),
        # the buffer that the grouped cast quantizes: 16384 rows of 5120 and their padding, 64 experts
        dict(name="dispatch_train", op="dispatch", T=4096, N=5120, E=64, k=4, dtype="bf16", align=128),
        # one token through a large projection: the weights are read once
        dict(name="linear_token", op="linear", T=1, N=14336, K=4096, dtype="bf16", out="bf16", bias=False),
        # a small batch, nothing a multiple of anything
        dict(name="linear_odd", op="linear", T=77, N=1000, K=1111, dtype="f32", out="f32", bias=True),
        # a long prompt through a large projection
        dict(name="linear_prompt", op="linear", T=8192, N=8192, K=8192, dtype="bf16", out="bf16", bias=False),
        # a decode batch through the experts: a few rows for each
        dict(name="experts_decode", op="experts", T=32, N=2048, K=5120, E=64, k=4, dtype="bf16", align=1),
        # a long prompt through the experts, the routed-expert shape of the contractions' workload
        dict(name="experts_prompt", op="experts", T=4096, N=2048, K=5120, E=64, k=4, dtype="bf16", align=128),
        # the expert rows of a decode batch back to its tokens
        dict(name="combine_decode", op="combine", T=32, N=5120, E=64, k=4, dtype="bf16", align=1, train=False),
        # the same of a training step, with the gradients of rows and weights
        dict(name="combine_train", op="combine", T=4096, N=5120, E=64, k=4, dtype="bf16", align=128, train=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "dispatch", "linear", "experts", "combine"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "linear":
        T, N, K = _log(rng, 1, 8192), _log(rng, 16, 14336), _log(rng, 16, 8192)
        return dict(op=op, T=T, N=N, K=K, dtype=dtype, out=rng.choice(["bf16", "f32"]), bias=rng.random() < 0.5)
    E = _log(rng, 4, 256 if op == "route" else 64)
    k = rng.randint(1, min(8, E))
    align = rng.choice([1, 16, 128])
    if op == "route":
        return dict(op=op, T=_log(rng, 1, 131072), E=E, k=k, dtype=dtype, align=align, train=rng.random() < 0.5,
                    normalize=rng.random() < 0.5)
    T = _log(rng, 1, 16384 // k)
    if op == "experts":
        return dict(op=op, T=T, N=_log(rng, 64, 2048), K=_log(rng, 64, 5120), E=E, k=k, dtype=dtype, align=align)
    case = dict(op=op, T=T, N=_log(rng, 16, 5120), E=E, k=k, dtype=dtype, align=align)
    if op == "combine":
        case["train"] = rng.random() < 0.5
    return case


def _rows(case):
    """Rows of the padded buffer: enough for every group's padding, whole groups of `align`."""
    picks, a = case["T"] * case["k"], case["align"]
    return -(-(picks + min(case["E"], picks) * (a - 1)) // a) * a


def work(case):
    op, T, esz = case["op"], case["T"], 2 if case["dtype"] == "bf16" else 4
    if op == "linear":
        N, K, osz = case["N"], case["K"], 2 if case["out"] == "bf16" else 4
        return {"bytes": T * K * esz + N * K + 4 * N * (2 if case["bias"] else 1) + T * N * osz, "flops": 2 * T * N * K}
    E, k, M = case["E"], case["k"], _rows(case)
    if op == "route":
        # logits, valid; idx, weight and slot of each pick, the row map, per-expert results; the gradient's dweight
        # and dlogits
        b = T * E * esz + T + 12 * T * k + 4 * M + 12 * E
        f = 5 * T * E
        if case["train"]:
            b += T * E * esz + 4 * T * k
            f += 4 * T * E
        return {"bytes": b, "flops": f}
    N = case["N"]
    if op == "dispatch":
        return {"bytes": T * N * esz + M * N * esz + 4 * T * k + 4 * M, "flops": 0}
    if op == "combine":
        b = T * k * N * esz + T * N * esz + 8 * T * k
        f = 2 * T * k * N
        if case["train"]:   # dy read, drows and dweight written
            b += T * N * esz + M * N * esz + 4 * T * k + 4 * M
            f += 3 * T * k * N
        return {"bytes": b, "flops": f}
    K = case["K"]
    # experts that get a token at all (uneven routing touches somewhat fewer)
    used = E * (1 - math.exp(-T * k / E))
    return {"bytes": int(T * K * esz + used * N * (K + 4) + M * N * 2 + 4 * T * k + 4 * M),
            "flops": 2 * T * k * N * K}


# --------------------------------------------------------------------------------------------------------- inputs
def _logits(case, g):
    """Router scores: some experts are liked more than others; a few tokens are barred from a few experts."""
    T, E = case["T"], case["E"]
    z = torch.randn(T, E, generator=g, device=DEV) * 1.5 + torch.randn(E, generator=g, device=DEV) * 0.5
    barred = torch.rand(T, E, generator=g, device=DEV) < 0.01
    return z.masked_fill(barred, -math.inf).to(DTYPES[case["dtype"]])


def _activations(T, K, g):
    """Hidden states: unit scale, every token its own size, a few channels much larger than the others."""
    x = torch.randn(T, K, generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn(T, 1, generator=g, device=DEV))
    return x * (1 + 15 * (torch.rand(K, generator=g, device=DEV) < 0.002))


def _weights8(shape, g):
    """Weights as a program keeps them: int8 codes [..., N, K] and a scale for each output channel."""
    w = torch.randn(*shape, generator=g, device=DEV) / math.sqrt(shape[-1])
    s = w.abs().amax(-1) / 127
    return torch.round(w / s[..., None]).clamp_(-127, 127).to(torch.int8), s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, T, dt = case["op"], case["T"], DTYPES[case["dtype"]]
    st = {"case": case}
    if op == "linear":
        st["x"] = _activations(T, case["K"], g).to(dt)
        st["B"], st["sB"] = _weights8((case["N"], case["K"]), g)
        st["bias"] = torch.randn(case["N"], generator=g, device=DEV) * 0.1 if case["bias"] else None
        st["out_dtype"] = DTYPES[case["out"]]
        return st
    E, k, M = case["E"], case["k"], _rows(case)
    st["logits"] = _logits(case, g)
    if op == "route":
        st["valid"] = torch.rand(T, generator=g, device=DEV) >= 0.02 if T > 1 else torch.ones(1, dtype=torch.bool, device=DEV)
        st["logits"].masked_fill_(~st["valid"][:, None], math.nan)
        st["dweight"] = torch.randn(T, k, generator=g, device=DEV)
        st["dloss"] = torch.full((1,), 0.01, device=DEV)
        if own:
            import mx9_dual_axis_amd as mxq

            st["plan"] = mxq.mx_routing(T, E, k, align=case["align"], device=DEV)
        return st
    valid = torch.ones(T, dtype=torch.bool, device=DEV)
    r = _route(st["logits"], valid, k, case["align"], M, True)
    st.update(slot=r["slot"], src=r["src"], offs=r["offs"], weight=r["weight"])
    if op == "dispatch":
        st["x"] = _activations(T, case["N"], g).to(dt)
    elif op == "combine":
        st["rows"] = torch.randn(M, case["N"], generator=g, device=DEV).to(dt)
        st["dy"] = torch.randn(T, case["N"], generator=g, device=DEV).to(dt)
    else:
        st["x"] = _activations(T, case["K"], g).to(dt)
        st["B"], st["sB"] = _weights8((E, case["N"], case["K"]), g)
        st["cap"] = int(r["counts"].max())   # the plain form's batched product needs the largest group's size
    return st


# ---------------------------------------------------------------------------------------------------- plain forms
def _live(z, valid):
    return valid & (z > -math.inf).any(1)


def _route(logits, valid, k, align, M, normalize):
    T, E = logits.shape
    z = logits.float().masked_fill(~valid[:, None], -math.inf)
    live = _live(z, valid)
    top = torch.where(live, z.amax(1), 0.0)
    e = torch.exp(z - top[:, None])
    p = torch.where(live[:, None], e / e.sum(1, keepdim=True), 0.0)
    val, idx = torch.sort(z, dim=1, descending=True, stable=True)   # equal scores: the lowest expert first
    val, idx = val[:, :k], idx[:, :k]
    ok = val > -math.inf
    w = torch.where(ok, p.gather(1, idx), 0.0)
    if normalize:
        w = w / torch.where(live, w.sum(1), 1.0)[:, None]
    chosen = torch.zeros(T, E, dtype=torch.int32, device=DEV).scatter_(1, idx, ok.to(torch.int32))
    before = torch.cumsum(chosen.t().contiguous(), 1, dtype=torch.int32).t() - chosen
    counts = chosen.sum(0, dtype=torch.int32)
    padded = (counts + (align - 1)) // align * align
    offs = torch.cumsum(padded, 0, dtype=torch.int32)
    slot = torch.where(ok, (offs - padded)[idx] + before.gather(1, idx), -1)
    src = torch.full((M + 1,), -1, dtype=torch.int32, device=DEV)
    src[torch.where(ok, slot, M).long().reshape(-1)] = torch.arange(T * k, dtype=torch.int32, device=DEV)
    n = live.sum(dtype=torch.int32).reshape(1)
    nf = n.clamp(min=1).float()
    prob = p.sum(0) / nf
    loss = E * (counts.float() / (k * nf) * prob).sum().reshape(1)
    return dict(idx=torch.where(ok, idx, -1).to(torch.int32), weight=w, slot=slot.to(torch.int32), src=src[:M],
                counts=counts, offs=offs, live=n, prob=prob, loss=loss)


def _route_grad(logits, valid, r, dweight, dloss, normalize):
    T, E = logits.shape
    k = dweight.shape[1]
    z = logits.float().masked_fill(~valid[:, None], -math.inf)
    live = _live(z, valid)[:, None]
    e = torch.exp(z - torch.where(live, z.amax(1, keepdim=True), 0.0))
    p = torch.where(live, e / e.sum(1, keepdim=True), 0.0)
    n = r["live"].clamp(min=1).float()
    g = (dloss * E * r["counts"].float() / (k * n * n)).expand(T, E)
    ok = r["idx"] >= 0
    at = r["idx"].clamp(min=0).long()
    dw = torch.where(ok, dweight, 0.0)
    if normalize:
        straight = r["weight"] * (dw - (r["weight"] * dw).sum(1, keepdim=True))
        d = p * (g - (p * g).sum(1, keepdim=True))
        d = d.scatter_add(1, at, torch.where(ok, straight, 0.0))
    else:
        g = g.scatter_add(1, at, dw)
        d = p * (g - (p * g).sum(1, keepdim=True))
    return d.to(logits.dtype)


def _quantize(x):
    a = x.abs().amax(1, keepdim=True).clamp(min=127 * 2.0**-126)
    return torch.round(x * (127 / a)), a / 127


def _rows_of(x, src, k):
    """Each row of the padded buffer: its token's row, or zeros."""
    return torch.where((src >= 0)[:, None], x[(src.clamp(min=0) // k).long()], torch.zeros((), dtype=x.dtype, device=DEV))


def _experts(st):
    case, offs = st["case"], st["offs"].long()
    M, E, cap = st["src"].numel(), case["E"], st["cap"]
    q, s = _quantize(_rows_of(st["x"].float(), st["src"], case["k"]))
    start = torch.cat([offs.new_zeros(1), offs[:-1]])
    at = start[:, None] + torch.arange(cap, device=DEV)
    inside = at < offs[:, None]
    a = q[torch.where(inside, at, 0)]
    c = torch.bmm(a, st["B"].float().transpose(1, 2).contiguous()) * st["sB"][:, None, :]
    out = torch.zeros(M + 1, case["N"], device=DEV)
    out[torch.where(inside, at, M)] = c
    return (out[:M] * s).to(torch.bfloat16)


def _run_plain(st):
    case, op = st["case"], st["case"]["op"]
    if op == "route":
        r = _route(st["logits"], st["valid"], case["k"], case["align"], _rows(case), case["normalize"])
        if case["train"]:
            r["dlogits"] = _route_grad(st["logits"], st["valid"], r, st["dweight"], st["dloss"], case["normalize"])
        return r
    if op == "linear":
        q, s = _quantize(st["x"].float())
        c = torch.matmul(q, st["B"].float().t()) * s * st["sB"]
        if st["bias"] is not None:
            c = c + st["bias"]
        return c.to(st["out_dtype"])
    if op == "dispatch":
        return _rows_of(st["x"], st["src"], case["k"])
    if op == "experts":
        return _experts(st)
    ok = st["slot"] >= 0
    w = torch.where(ok, st["weight"], 0.0)
    rows = torch.where(ok[..., None], st["rows"].float()[st["slot"].clamp(min=0).long()], 0.0)
    out = {"y": (w[..., None] * rows).sum(1).to(st["rows"].dtype)}
    if case["train"]:
        dy, src = st["dy"].float(), st["src"]
        pick = src.clamp(min=0).long()
        d = dy[pick // case["k"]] * w.reshape(-1)[pick][:, None]
        out["drows"] = torch.where((src >= 0)[:, None], d, 0.0).to(st["rows"].dtype)
        out["dweight"] = (dy[:, None, :] * rows).sum(2)
    return out


def _run_own(st):
    import mx9_dual_axis_amd as mxq

    case, op = st["case"], st["case"]["op"]
    if op == "route":
        r = mxq.mx_route(st["logits"], case["k"], valid=st["valid"], normalize=case["normalize"], out=st["plan"])
        out = dict(idx=r.idx, weight=r.weight, slot=r.slot, src=r.src, counts=r.counts, offs=r.offs, live=r.live,
                   prob=r.prob, loss=r.loss)
        if case["train"]:
            out["dlogits"] = mxq.mx_route_grad(st["logits"], r, dweight=st["dweight"], dloss=st["dloss"], valid=st["valid"])
        return out
    if op == "linear":
        return mxq.i8_linear(st["x"], st["B"], st["sB"], bias=st["bias"], out_dtype=st["out_dtype"])
    if op == "dispatch":
        return mxq.mx_dispatch(st["x"], st["slot"], st["src"])
    if op == "experts":
        q, s = mxq.mx_dispatch_i8(st["x"], st["slot"], st["src"])
        return mxq.i8_grouped_gemm_rows(q, s, st["B"], st["sB"], st["offs"], out_dtype=torch.bfloat16)
    out = {"y": mxq.mx_combine(st["rows"], st["slot"], st["weight"])}
    if case["train"]:
        out["drows"], out["dweight"] = mxq.mx_combine_grad(st["dy"], st["rows"], st["slot"], st["weight"], st["src"])
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# --------------------------------------------------------------------------------------- the definitions, 64 bits
def _exact_route(st):
    case = st["case"]
    T, E, k = case["T"], case["E"], case["k"]
    z = st["logits"].double()
    z[~st["valid"]] = -math.inf
    chosen = torch.empty(T, E, dtype=torch.bool, device=DEV)
    lower = torch.ones(E, E, dtype=torch.bool, device=DEV).tril(-1)      # [e, f]: f < e
    for t in range(0, T, 1024):
        a, b = z[t:t + 1024, :, None], z[t:t + 1024, None, :]
        place = (b > a).sum(2) + ((b == a) & lower).sum(2)               # experts that come before e
        chosen[t:t + 1024] = (place < k) & (z[t:t + 1024] > -math.inf)
    alive = torch.isfinite(z).any(1)
    n = max(1, int(alive.sum()))
    p = torch.zeros_like(z)
    p[alive] = torch.softmax(z[alive], 1)
    count = chosen.sum(0).double()
    mean = p.sum(0) / n
    val = torch.topk(z, k, dim=1).values                                # values do not depend on the order of ties
    w = torch.zeros(T, k, dtype=torch.float64, device=DEV)
    w[alive] = torch.exp(val[alive] - torch.logsumexp(z[alive], 1, keepdim=True))
    if case["normalize"]:
        w[alive] = torch.softmax(val[alive], 1)
    out = dict(idx=None, weight=w, slot=None, src=None, counts=None, offs=None, live=None, prob=mean,
               loss=(E * (count * mean).sum() / (k * n)).reshape(1))
    if case["train"]:
        # picks in the order of the weights: descending score, lowest expert first
        order = torch.sort(torch.where(chosen, z, -math.inf), dim=1, descending=True, stable=True).indices[:, :k]
        real = chosen.gather(1, order)
        dw = torch.where(real, st["dweight"].double(), 0.0)
        up = torch.zeros(T, E, dtype=torch.float64, device=DEV)
        up.scatter_add_(1, order, dw)                                   # dL/d(weight) by expert
        a = st["dloss"].double() * E * count / (k * n) / n              # dL/dp of the balance loss
        if case["normalize"]:
            v = torch.zeros_like(up)
            v.scatter_add_(1, order, torch.where(real, w, 0.0))
            d = v * (up - (v * up).sum(1, keepdim=True)) + p * (a - (p @ a)[:, None])
        else:
            a = a + up
            d = p * (a - (p * a).sum(1, keepdim=True))
        d[~alive] = 0.0
        out["dlogits"] = d
    return out


def _exact_codes(x):
    """Codes and scales of rows that all have a nonzero element of ordinary size."""
    s = x.abs().amax(1) / 127
    return torch.round(x / s[:, None]), s


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(st)
    if op == "linear":
        q, s = _exact_codes(st["x"].double())
        c = (q * s[:, None]) @ (st["B"].double() * st["sB"].double()[:, None]).t().contiguous()
        return c + st["bias"].double() if st["bias"] is not None else c
    if op == "dispatch":
        out = torch.zeros(st["src"].numel(), case["N"], dtype=torch.float64, device=DEV)
        for j in range(case["k"]):
            t = (st["slot"][:, j] >= 0).nonzero()[:, 0]
            out[st["slot"][t, j].long()] = st["x"][t].double()
        return out
    if op == "experts":
        q, s = _exact_codes(st["x"].double())
        c = torch.zeros(st["src"].numel(), case["N"], dtype=torch.float64, device=DEV)
        ends = [0] + st["offs"].tolist()
        pick = st["src"].long()
        for e in range(case["E"]):
            rows = torch.arange(ends[e], ends[e + 1], device=DEV)
            rows = rows[pick[rows] >= 0]
            if rows.numel():
                t = pick[rows] // case["k"]
                c[rows] = (q[t] * s[t, None]) @ (st["B"][e].double() * st["sB"][e].double()[:, None]).t().contiguous()
        return c
    T, k, N = case["T"], case["k"], case["N"]
    y = torch.zeros(T, N, dtype=torch.float64, device=DEV)
    drows = torch.zeros(st["src"].numel(), N, dtype=torch.float64, device=DEV)
    dweight = torch.zeros(T, k, dtype=torch.float64, device=DEV)
    dy, w = st["dy"].double(), st["weight"].double()
    for j in range(k):
        t = (st["slot"][:, j] >= 0).nonzero()[:, 0]
        at = st["slot"][t, j].long()
        r = st["rows"][at].double()
        y[t] += w[t, j, None] * r
        drows[at] = w[t, j, None] * dy[t]
        dweight[t, j] = (dy[t] * r).sum(1)
    return dict(y=y, drows=drows, dweight=dweight) if case["train"] else dict(y=y)
