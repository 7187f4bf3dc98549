"""What is measured of scored routing and of the products with an epilogue.

The operators, and the calls that run them:
  scored routing   mx_route_scored, mx_route_scored_grad, mx_route_bias_step: sigmoid or softmax scores, the k best
                   experts by score plus a balancing bias out of the best groups of experts, weights by the scores
                   alone; counts, padded group ends, row map and balance loss as of the other routing; the gradient
                   of weights and loss; the bias's step towards even counts
  8-bit product    i8_linear_act, i8_grouped_gemm_rows_act: the product of 8-bit integer codes, dense and by expert,
                   with bias, activation (plain, or of the first half of the channels times the second) and residual
                   applied before the only rounding
  MXFP8 product    mx_gemm_nt_act, mx_grouped_gemm_rows_act: the same on the MXFP8 contraction, which can keep the
                   values before the activation for the backward pass
  epilogue's grad  mx_act_grad: the gradient of those values, and of the bias (by expert where there are groups)

Scores are compared in 64 bits: equal ones go to the lowest expert.  A logit of -inf is an expert that the token may
not use; a token that is not valid may hold anything.  Rows behind the last group give 0.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"
EPS = 1e-20               # added to the sums that scores are divided by


# ---------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one token of one sequence while it is being decoded: sigmoid scores, half of the groups stay
        dict(name="route_token", op="route", T=1, E=256, k=8, groups=8, top=4, best=2, score="sigmoid", bias=True,
             normalize=True, scale=2.5, dtype="bf16", align=1, train=False),
        # a small ragged training batch: softmax scores, the best expert stands for its group, weights as they are
        dict(name="route_odd", op="route", T=777, E=60, k=6, groups=4, top=2, best=1, score="softmax", bias=True,
             normalize=False, scale=1.0, dtype="bf16", align=16, train=True),
        # a long-sequence training batch over many experts, scores kept in fp32
        dict(name="route_large", op="route", T=131072, E=256, k=8, groups=8, top=4, best=2, score="sigmoid", bias=True,
             normalize=True, scale=2.5, dtype="f32", align=128, train=True),
        # one token through the gated projection of a feed-forward layer: the weights are read once
        dict(name="i8_token", op="i8", T=1, N=7168, K=4096, act="silu", gated=True, bias=False, residual=False,
             dtype="bf16"),
        # a small batch, nothing a multiple of anything, fp32 throughout
        dict(name="i8_odd", op="i8", T=77, N=1000, K=1111, act="gelu", gated=False, bias=True, residual=True,
             dtype="f32"),
        # a long prompt through a large projection
        dict(name="i8_prompt", op="i8", T=8192, N=8192, K=8192, act="gelu_tanh", gated=False, bias=True, residual=True,
             dtype="bf16"),
        # a decode batch through the experts' gated projections: a few rows for each
        dict(name="i8_experts", op="i8_experts", T=32, N=1024, K=5120, E=64, k=4, act="silu", gated=True, bias=False,
             dtype="bf16", align=1),
        # the smallest training batch of a dense layer
        dict(name="mx_small", op="mx", M=128, N=5120, K=5120, act="silu", gated=False, bias=True, residual=True,
             keep=True),
        # a large dense layer in training, whose backward needs the values before the activation
        dict(name="mx_dense", op="mx", M=8192, N=8192, K=8192, act="gelu", gated=False, bias=True, residual=True,
             keep=True),
        # the experts' gated projections in training
        dict(name="mx_experts", op="mx_experts", T=4096, N=1024, K=5120, E=64, k=4, act="silu", gated=True, bias=True,
             keep=True, align=128),
        # the backward of a small odd layer in fp32
        dict(name="grad_odd", op="grad", M=333, N=1111, act="gelu", gated=False, bias=True, dtype="f32"),
        # the backward of the experts' gated projections: a bias for each expert
        dict(name="grad_experts", op="grad_experts", T=4096, N=2048, E=64, k=4, act="silu", gated=True, bias=True,
             dtype="bf16", align=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route", "i8", "i8_experts", "mx", "mx_experts", "grad", "grad_experts"])
    act = rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"])
    gated, bias, residual = rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.5
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "route":
        groups = rng.choice([1, 2, 3, 4, 8])
        size = _log(rng, 4, 256 // groups)
        top = rng.randint(1, groups)
        return dict(op=op, T=_log(rng, 1, 131072), E=groups * size, k=rng.randint(1, min(8, top * size)), groups=groups,
                    top=top, best=rng.choice([1, 2]), score=rng.choice(["sigmoid", "softmax"]), bias=bias,
                    normalize=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]), dtype=dtype,
                    align=rng.choice([1, 16, 128]), train=rng.random() < 0.5)
    if op == "i8":
        return dict(op=op, T=_log(rng, 1, 8192), N=_log(rng, 16, 7168), K=_log(rng, 16, 8192), act=act, gated=gated,
                    bias=bias, residual=residual, dtype=dtype)
    if op == "mx":
        return dict(op=op, M=128 * _log(rng, 1, 64), N=128 * _log(rng, 1, 32), K=128 * _log(rng, 1, 64), act=act,
                    gated=gated, bias=bias, residual=residual, keep=rng.random() < 0.5)
    if op == "grad":
        return dict(op=op, M=_log(rng, 1, 24576), N=_log(rng, 16, 4096), act=act, gated=gated, bias=bias, dtype=dtype)
    E = _log(rng, 4, 64)
    k = rng.randint(1, min(4, E))
    case = dict(op=op, T=_log(rng, 1, 4096), E=E, k=k, act=act, gated=gated, bias=bias)
    if op == "i8_experts":
        return dict(case, N=_log(rng, 64, 1024), K=_log(rng, 64, 5120), dtype=dtype, align=rng.choice([1, 16, 128]))
    if op == "mx_experts":
        return dict(case, N=128 * rng.randint(1, 8), K=128 * _log(rng, 1, 40), keep=rng.random() < 0.5, align=128)
    return dict(case, N=_log(rng, 64, 2048), dtype=dtype, align=rng.choice([1, 16, 128]))


def _rows(case):
    """Rows of the padded buffer: enough for every group's padding, whole groups of `align`."""
    picks, a = case["T"] * case["k"], case["align"]
    return -(-(picks + min(case["E"], picks) * (a - 1)) // a) * a


def work(case):
    op = case["op"]
    if op == "route":
        T, E, k, M = case["T"], case["E"], case["k"], _rows(case)
        esz = 2 if case["dtype"] == "bf16" else 4
        b = T * E * esz + T + 12 * T * k + 4 * M + 12 * E + (4 * E if case["bias"] else 0)
        f = 6 * T * E
        if case["train"]:   # the gradient's dweight and dlogits; the bias's step
            b += T * E * esz + 4 * T * k + (4 * E if case["bias"] else 0)
            f += 4 * T * E
        return {"bytes": b, "flops": f}
    N, W = case["N"], case["N"] * (2 if case["gated"] else 1)     # results and channels of a row
    if op in ("grad", "grad_experts"):
        esz, M = 2 if case["dtype"] == "bf16" else 4, case["M"] if op == "grad" else _rows(case)
        sums = (1 if op == "grad" else case["E"]) * W * 4 if case["bias"] else 0
        return {"bytes": M * N * esz + 2 * M * W * esz + sums, "flops": 12 * M * W}
    K = case["K"]
    if op == "i8":
        T, esz = case["T"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": T * K * esz + W * K + 4 * W * (2 if case["bias"] else 1) + T * N * esz * (2 if case["residual"] else 1),
                "flops": 2 * T * W * K}
    if op == "mx":
        M = case["M"]
        out = M * N * 2 * (2 if case["residual"] else 1) + (M * W * 2 if case["keep"] else 0)
        return {"bytes": (M + W) * K * 33 // 32 + (4 * W if case["bias"] else 0) + out, "flops": 2 * M * W * K}
    # by expert: experts that get a token at all (uneven groups touch somewhat fewer)
    T, k, M, E = case["T"], case["k"], _rows(case), case["E"]
    used = E * (1 - math.exp(-T * k / E))
    if op == "i8_experts":
        esz = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": int(T * k * (K + 4) + used * W * (K + (8 if case["bias"] else 4)) + M * N * esz), "flops": 2 * T * k * W * K}
    out = M * N * 2 + (M * W * 2 if case["keep"] else 0)
    return {"bytes": int((T * k + used * W) * K * 33 / 32 + (used * 4 * W if case["bias"] else 0) + out), "flops": 2 * T * k * W * K}


# --------------------------------------------------------------------------------------------------------- inputs
def _activations(T, K, g):
    """Hidden states: unit scale, every token its own size, a few channels much larger than the others."""
    x = torch.randn(T, K, generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn(T, 1, generator=g, device=DEV))
    return x * (1 + 15 * (torch.rand(K, generator=g, device=DEV) < 0.002))


def _codes8(w):
    """int8 codes of the rows and a scale for each."""
    s = w.abs().amax(-1).clamp(min=127 * 2.0 ** -126) / 127
    return torch.round(w / s[..., None]).clamp_(-127, 127).to(torch.int8), s


def _codes_mx(w):
    """E4M3 codes (as bytes) of the rows and an E8M0 scale for each 32 of a row."""
    b = w.reshape(*w.shape[:-1], w.shape[-1] // 32, 32)
    e = torch.frexp(b.abs().amax(-1)).exponent.clamp(-100, 100) - 8      # the largest below 2^8, under e4m3's 448
    q = (b * torch.exp2(-e.float())[..., None]).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).reshape(w.shape), (e + 127).to(torch.uint8)


def _weights(shape, codes, g):
    """Weights by output channel, a matrix of them at a time."""
    if len(shape) == 2:
        return codes(torch.randn(*shape, generator=g, device=DEV) / math.sqrt(shape[-1]))
    parts = [codes(torch.randn(*shape[1:], generator=g, device=DEV) / math.sqrt(shape[-1])) for _ in range(shape[0])]
    return torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])


def _grouped_rows(case, g):
    """Rows of uneven groups: their number in each, the groups' padded ends, which rows hold a token."""
    T, E, k, align, M = case["T"], case["E"], case["k"], case["align"], _rows(case)
    liked = torch.randn(E, generator=g, device=DEV) * 0.6
    score = torch.rand(T, E, generator=g, device=DEV).log().neg().log().neg() + liked
    counts = torch.bincount(score.topk(k, dim=1).indices.reshape(-1), minlength=E)
    padded = (counts + (align - 1)) // align * align
    offs = padded.cumsum(0)
    at = torch.arange(M, device=DEV)
    e = torch.searchsorted(offs, at, right=True)
    inside = e < E
    e = e.clamp(max=E - 1)
    return counts, offs.to(torch.int32), inside & (at - (offs - padded)[e] < counts[e])


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    op, st = case["op"], {"case": case}
    if op == "route":
        T, E, k, dt = case["T"], case["E"], case["k"], DTYPES[case["dtype"]]
        z = rnd(T, E) * 1.5 + rnd(E) * 0.5
        z = z.masked_fill(torch.rand(T, E, generator=g, device=DEV) < 0.01, -math.inf).to(dt)
        valid = torch.rand(T, generator=g, device=DEV) >= 0.02 if T > 1 else torch.ones(1, dtype=torch.bool, device=DEV)
        st["logits"] = z.masked_fill(~valid[:, None], math.nan)
        st["valid"] = valid
        st["bias"] = rnd(E) * 0.05 if case["bias"] else None
        st["dweight"], st["dloss"] = rnd(T, k), torch.full((1,), 0.01, device=DEV)
        if own:
            import mx9_dual_axis_amd as mxq

            st["plan"] = mxq.mx_routing(T, E, k, align=case["align"], device=DEV)
        return st
    N, W = case["N"], case["N"] * (2 if case["gated"] else 1)
    grouped = op.endswith("experts")
    if grouped:
        counts, st["offs"], real = _grouped_rows(case, g)
        st["cap"] = int(counts.max())      # the plain form's batched product needs the largest group's size
    E = case["E"] if grouped else 1
    if op in ("grad", "grad_experts"):
        M, dt = case["M"] if op == "grad" else _rows(case), DTYPES[case["dtype"]]
        st["dy"], st["pre"] = rnd(M, N), rnd(M, W) * 1.5
        if grouped:
            st["dy"] *= real[:, None]
        st["dy"], st["pre"] = st["dy"].to(dt), st["pre"].to(dt)
        return st
    K = case["K"]
    st["bias"] = (rnd(E, W) if grouped else rnd(W)) * 0.1 if case["bias"] else None
    rows = _rows(case) if grouped else case["T"] if op == "i8" else case["M"]
    x = _activations(rows, K, g)
    if grouped:
        x *= real[:, None]
    if op.startswith("i8"):
        dt = DTYPES[case["dtype"]]
        if grouped:
            st["x"], st["sx"] = _codes8(x)
        else:
            st["x"] = x.to(dt)
        st["B"], st["sB"] = _weights((E, W, K) if grouped else (W, K), _codes8, g)
    else:
        dt = torch.bfloat16
        st["x"], st["sx"] = _codes_mx(x)
        st["B"], st["sB"] = _weights((E, W, K) if grouped else (W, K), _codes_mx, g)
    st["residual"] = rnd(rows, N).to(dt) if case.get("residual") else None
    st["out_dtype"] = dt
    return st


# ---------------------------------------------------------------------------------------------------- plain forms
def _scores(z, live, kind):
    if kind == "sigmoid":
        return torch.where(live, 1 / (1 + torch.exp(-z)), 0.0)
    e = torch.exp(z - torch.where(live, z.amax(1, keepdim=True), 0.0))
    return torch.where(live, e / e.sum(1, keepdim=True), 0.0)


def _select(z, s, bias, case):
    """The picks' experts (and which of them are any), from scores in 64 bits."""
    T, E = z.shape
    G, k = case["groups"], case["k"]
    u = torch.where(z > -math.inf, s + bias if bias is not None else s, -math.inf)
    if G > 1:
        two = torch.sort(u.view(T, G, E // G), dim=2, descending=True).values[:, :, :case["best"]]
        worth = two[:, :, 0] + torch.where(two[:, :, 1:] > -math.inf, two[:, :, 1:], 0.0).sum(2)
        order = torch.sort(worth, dim=1, descending=True, stable=True).indices[:, :case["top"]]
        stays = torch.zeros(T, G, dtype=torch.bool, device=DEV).scatter_(1, order, True)
        stays = stays.repeat_interleave(E // G, dim=1)
    else:
        stays = torch.ones((), dtype=torch.bool, device=DEV)
    u = torch.where(stays, u if bias is not None else z, -math.inf)   # without a bias the logits have the scores' order
    val, idx = torch.sort(u, dim=1, descending=True, stable=True)
    return idx[:, :k], val[:, :k] > -math.inf


def _route(st):
    case, valid = st["case"], st["valid"]
    T, E = st["logits"].shape
    k, align, M = case["k"], case["align"], _rows(case)
    z64 = st["logits"].double().masked_fill(~valid[:, None], -math.inf)
    live = (z64 > -math.inf).any(1, keepdim=True)
    bias = st["bias"]
    idx, ok = _select(z64, _scores(z64, live, case["score"]), None if bias is None else bias.double(), case)
    s = _scores(z64.float(), live, case["score"])
    w = torch.where(ok, s.gather(1, idx), 0.0)
    if case["normalize"]:
        w = w / (w.sum(1, keepdim=True) + EPS)
    w = w * case["scale"]
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
    share = s / (s.sum(1, keepdim=True) + EPS) if case["score"] == "sigmoid" else s
    prob = share.sum(0) / nf
    loss = E * (counts.float() / (k * nf) * prob).sum().reshape(1)
    return dict(idx=torch.where(ok, idx, -1).to(torch.int32), weight=w, slot=slot.to(torch.int32), src=src[:M],
                counts=counts, offs=offs, live=n, prob=prob, loss=loss)


def _route_grad(st, r):
    case = st["case"]
    E, k = case["E"], case["k"]
    z = st["logits"].float().masked_fill(~st["valid"][:, None], -math.inf)
    live = (z > -math.inf).any(1, keepdim=True)
    s = _scores(z, live, case["score"])
    n = r["live"].clamp(min=1).float()
    a = st["dloss"] * E * r["counts"].float() / (k * n * n)
    ok = r["idx"] >= 0
    at = r["idx"].clamp(min=0).long()
    d = torch.where(ok, st["dweight"], 0.0) * case["scale"]
    if case["normalize"]:
        sj = torch.where(ok, s.gather(1, at), 0.0)
        q = 1 / (sj.sum(1, keepdim=True) + EPS)
        d = torch.where(ok, q * (d - q * (d * sj).sum(1, keepdim=True)), 0.0)
    if case["score"] == "sigmoid":
        q = 1 / (s.sum(1, keepdim=True) + EPS)
        ds = q * (a - q * (a * s).sum(1, keepdim=True))
        out = ds.scatter_add(1, at, d) * s * (1 / (1 + torch.exp(z)))
    else:
        # the picks' part apart from the loss's, which is much smaller
        part = s.gather(1, at) * d
        out = s * (a - (s * a).sum(1, keepdim=True)) - s * part.sum(1, keepdim=True)
        out = out.scatter_add(1, at, part)
    return torch.where(live, out, 0.0).to(st["logits"].dtype)


def _act(x, act):
    if act == "relu":
        return torch.where(x > 0, x, 0.0)
    if act == "silu":
        return x / (1 + torch.exp(-x))
    if act == "gelu":
        return x * (0.5 * torch.erfc(x * -math.sqrt(0.5)))
    if act == "gelu_tanh":
        return x / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))
    return x


def _act_slope(x, act):
    if act == "relu":
        return (x > 0).to(x.dtype)
    if act == "silu":
        p = 1 / (1 + torch.exp(-x))
        return p * (1 + x / (1 + torch.exp(x)))
    if act == "gelu":
        return 0.5 * torch.erfc(x * -math.sqrt(0.5)) + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        t = c * (x + 0.044715 * x * x * x)
        p = 1 / (1 + torch.exp(-t))
        return p * (1 + x / (1 + torch.exp(t)) * c * (1 + 3 * 0.044715 * x * x))
    return torch.ones_like(x)


def _epilogue(c, case, residual):
    """(results, the values before the activation) of sums with their bias in fp32."""
    if case["gated"]:
        gate, up = c.chunk(2, dim=1)
        y = _act(gate, case["act"]) * up
    else:
        y = _act(c, case["act"])
    return y if residual is None else y + residual.float()


def _quantize(x):
    a = x.abs().amax(1, keepdim=True).clamp(min=127 * 2.0**-126)
    return torch.round(x * (127 / a)), a / 127


def _mx_values(q, s):
    w = q.view(torch.float8_e4m3fn).float()
    return (w.view(*s.shape, 32) * torch.exp2(s.float() - 127)[..., None]).view(q.shape)


def _groups(offs, M):
    """(first row, end) of each group."""
    offs = offs.long()
    return torch.cat([offs.new_zeros(1), offs[:-1]]), offs


def _by_expert(x, B, st, bias, sB):
    """Each group's rows times its expert's matrix (and its channels' scales), plus its bias; 0 behind the last group."""
    M, W = x.shape[0], B.shape[1]
    start, end = _groups(st["offs"], M)
    size = int(min(M, st["cap"] + st["case"]["align"]))
    at = start[:, None] + torch.arange(size, device=DEV)
    inside = at < end[:, None]
    a = x[torch.where(inside, at, 0)]
    c = torch.bmm(a, B.transpose(1, 2).contiguous())
    if sB is not None:
        c = c * sB[:, None, :]
    if bias is not None:
        c = c + bias[:, None, :]
    out = torch.zeros(M + 1, W, device=DEV)
    out[torch.where(inside, at, M)] = c
    return out[:M]


def _run_plain(st):
    case, op = st["case"], st["case"]["op"]
    if op == "route":
        r = _route(st)
        if case["train"]:
            r["dlogits"] = _route_grad(st, r)
            if st["bias"] is not None:
                c = r["counts"]
                r["next_bias"] = st["bias"] + 0.001 * torch.sign(c.sum() - c.long() * case["E"]).float()
        return r
    if op in ("grad", "grad_experts"):
        dy, pre = st["dy"].float(), st["pre"].float()
        M = pre.shape[0]
        start, end = _groups(st["offs"], M) if op == "grad_experts" else (None, None)
        if op == "grad_experts":
            dy = torch.where((torch.arange(M, device=DEV) < end[-1])[:, None], dy, 0.0)
        if case["gated"]:
            gate, up = pre.chunk(2, dim=1)
            d = torch.cat([dy * up * _act_slope(gate, case["act"]), dy * _act(gate, case["act"])], dim=1)
        else:
            d = dy * _act_slope(pre, case["act"])
        out = {"dpre": d.to(st["pre"].dtype)}
        if case["bias"]:
            if op == "grad":
                out["dbias"] = d.sum(0)
            else:
                e = torch.searchsorted(end, torch.arange(M, device=DEV), right=True)
                sums = torch.zeros(case["E"] + 1, d.shape[1], device=DEV)
                out["dbias"] = sums.index_add(0, e, d)[:case["E"]]
        return out
    if op == "i8":
        q, s = _quantize(st["x"].float())
        c = torch.matmul(q, st["B"].float().t()) * s * st["sB"]
        if st["bias"] is not None:
            c = c + st["bias"]
        return _epilogue(c, case, st["residual"]).to(st["out_dtype"])
    if op == "i8_experts":
        c = _by_expert(st["x"].float(), st["B"].float(), st, None, st["sB"]) * st["sx"][:, None]
        if st["bias"] is not None:
            e = torch.searchsorted(st["offs"].long(), torch.arange(c.shape[0], device=DEV), right=True)
            c = c + torch.cat([st["bias"], torch.zeros_like(st["bias"][:1])])[e]
        return _epilogue(c, case, None).to(st["out_dtype"])
    x, B = _mx_values(st["x"], st["sx"]), _mx_values(st["B"], st["sB"])
    if op == "mx":
        c = torch.matmul(x, B.t())
        if st["bias"] is not None:
            c = c + st["bias"]
    else:
        c = _by_expert(x, B, st, st["bias"], None)
    out = {"y": _epilogue(c, case, st["residual"]).to(torch.bfloat16)}
    if case["keep"]:
        out["pre"] = c.to(torch.bfloat16)
    return out


def _run_own(st):
    import mx9_dual_axis_amd as mxq

    case, op = st["case"], st["case"]["op"]
    if op == "route":
        r = mxq.mx_route_scored(st["logits"], bias=st["bias"], score=case["score"], groups=case["groups"],
                                top_groups=case["top"], group_best=case["best"], normalize=case["normalize"],
                                scale=case["scale"], valid=st["valid"], out=st["plan"])
        out = dict(idx=r.idx, weight=r.weight, slot=r.slot, src=r.src, counts=r.counts, offs=r.offs, live=r.live,
                   prob=r.prob, loss=r.loss)
        if case["train"]:
            out["dlogits"] = mxq.mx_route_scored_grad(st["logits"], r, dweight=st["dweight"], dloss=st["dloss"],
                                                      valid=st["valid"])
            if st["bias"] is not None:
                out["next_bias"] = mxq.mx_route_bias_step(st["bias"], r.counts, 0.001)
        return out
    act, gated = case["act"], case["gated"]
    if op in ("grad", "grad_experts"):
        dpre, dbias = mxq.mx_act_grad(st["dy"], st["pre"], act, gated, offs=st.get("offs"), bias=case["bias"])
        return {"dpre": dpre, "dbias": dbias} if case["bias"] else {"dpre": dpre}
    if op == "i8":
        return mxq.i8_linear_act(st["x"], st["B"], st["sB"], bias=st["bias"], act=act, gated=gated,
                                 residual=st["residual"], out_dtype=st["out_dtype"])
    if op == "i8_experts":
        return mxq.i8_grouped_gemm_rows_act(st["x"], st["sx"], st["B"], st["sB"], st["offs"], bias=st["bias"], act=act,
                                            gated=gated, out_dtype=st["out_dtype"])
    pre = True if case["keep"] else None
    if op == "mx":
        y = mxq.mx_gemm_nt_act(st["x"], st["sx"], st["B"], st["sB"], bias=st["bias"], act=act, gated=gated,
                               residual=st["residual"], out_dtype=torch.bfloat16, pre=pre)
    else:
        y = mxq.mx_grouped_gemm_rows_act(st["x"], st["sx"], st["B"], st["sB"], st["offs"], bias=st["bias"], act=act,
                                         gated=gated, out_dtype=torch.bfloat16, pre=pre)
    return {"y": y[0], "pre": y[1]} if case["keep"] else {"y": y}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# --------------------------------------------------------------------------------------- the definitions, 64 bits
def _exact_route(st):
    case = st["case"]
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    size = E // G
    z = st["logits"].double()
    z[~st["valid"]] = -math.inf
    alive = torch.isfinite(z).any(1)
    s = torch.zeros_like(z)
    s[alive] = torch.sigmoid(z[alive]) if case["score"] == "sigmoid" else torch.softmax(z[alive], 1)
    can = torch.isfinite(z)
    b = torch.zeros(E, dtype=torch.float64, device=DEV) if st["bias"] is None else st["bias"].double()
    u = s + b
    chosen = torch.zeros(T, E, dtype=torch.bool, device=DEV)
    lower = torch.ones(E, E, dtype=torch.bool, device=DEV).tril(-1)      # [e, f]: f < e
    for t in range(0, T, 1024):
        ut, ct = u[t:t + 1024].masked_fill(~can[t:t + 1024], -math.inf), can[t:t + 1024]
        if G > 1:
            grp = ut.view(-1, G, size)
            worth = grp.amax(2)
            if case["best"] == 2 and size > 1:
                second = torch.topk(grp, 2, dim=2).values[:, :, 1]
                worth = worth + second.masked_fill(second == -math.inf, 0.0)
            low = torch.ones(G, G, dtype=torch.bool, device=DEV).tril(-1)
            a, c = worth[:, :, None], worth[:, None, :]
            ahead = (c > a).sum(2) + ((c == a) & low).sum(2)
            ct = ct & (ahead < case["top"])[:, :, None].expand(-1, G, size).reshape(-1, E)
        v = (z[t:t + 1024] if st["bias"] is None else ut).masked_fill(~ct, -math.inf)
        a, c = v[:, :, None], v[:, None, :]
        chosen[t:t + 1024] = ((c > a).sum(2) + ((c == a) & lower).sum(2) < k) & ct
    n = max(1, int(alive.sum()))
    count = chosen.sum(0).double()
    picked = torch.where(chosen, u if st["bias"] is not None else z, -math.inf)
    order = torch.sort(picked, dim=1, descending=True, stable=True).indices[:, :k]
    real = chosen.gather(1, order)
    sj = torch.where(real, s.gather(1, order), 0.0)
    total = sj.sum(1, keepdim=True) + EPS
    w = case["scale"] * (sj / total if case["normalize"] else sj)
    mass = s.sum(1, keepdim=True) + EPS
    share = s / mass if case["score"] == "sigmoid" else s
    mean = share.sum(0) / n
    out = dict(idx=None, weight=w, slot=None, src=None, counts=None, offs=None, live=None, prob=mean,
               loss=(E * (count * mean).sum() / (k * n)).reshape(1))
    if not case["train"]:
        return out
    dw = torch.where(real, st["dweight"].double(), 0.0) * case["scale"]
    if case["normalize"]:
        dw = (dw - (dw * sj).sum(1, keepdim=True) / total) / total
        dw = torch.where(real, dw, 0.0)
    up = torch.zeros_like(z).scatter_add_(1, order, dw)                  # dL/ds by expert
    a = st["dloss"].double() * E * count / (k * n) / n                   # dL/d(share)
    if case["score"] == "sigmoid":
        ds = up + (a - (share @ a)[:, None]) / mass
        d = ds * s * torch.sigmoid(-z)
    else:
        ds = up + a
        d = s * (ds - (s * ds).sum(1, keepdim=True))
    d[~alive] = 0.0
    out["dlogits"] = d
    if st["bias"] is not None:
        out["next_bias"] = b + 0.001 * torch.sign(count.mean() - count)
    return out


def _exact_act(x, act):
    F = torch.nn.functional
    if act == "gelu":
        return x * torch.special.ndtr(x)
    return {"none": lambda v: v, "relu": F.relu, "silu": lambda v: v * torch.sigmoid(v),
            "gelu_tanh": lambda v: 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))}[act](x)


def _exact_epilogue(c, case, residual):
    N = case["N"]
    y = _exact_act(c[:, :N], case["act"]) * c[:, N:] if case["gated"] else _exact_act(c, case["act"])
    return y if residual is None else y + residual.double()


def _exact_mx(q, s):
    w = q.view(torch.float8_e4m3fn).double()
    return w * torch.exp2(s.double() - 127).repeat_interleave(32, dim=-1)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(st)
    N = case["N"]
    ends = [0] + st["offs"].tolist() if op.endswith("experts") else [0]
    if op in ("grad", "grad_experts"):
        dy, x = st["dy"].double(), st["pre"].double()
        if op == "grad_experts":
            dy[ends[-1]:] = 0.0
        if case["act"] == "gelu":                                       # its derivative by the normal density
            slope = lambda v: torch.special.ndtr(v) + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)  # noqa: E731
        else:
            def slope(v):
                v = v.clone().requires_grad_()
                return torch.autograd.grad(_exact_act(v, case["act"]).sum(), v)[0]
        if case["gated"]:
            gate, up = x[:, :N], x[:, N:]
            d = torch.cat([dy * up * slope(gate), dy * _exact_act(gate, case["act"])], dim=1)
        else:
            d = dy * slope(x)
        out = {"dpre": d}
        if case["bias"]:
            if op == "grad":
                out["dbias"] = d.sum(0)
            else:
                out["dbias"] = torch.stack([d[a:b].sum(0) for a, b in zip(ends, ends[1:])])
        return out
    if op == "i8":
        x = st["x"].double()
        s = x.abs().amax(1, keepdim=True) / 127
        c = (torch.round(x / s) * s) @ (st["B"].double() * st["sB"].double()[:, None]).t().contiguous()
        if st["bias"] is not None:
            c = c + st["bias"].double()
        return _exact_epilogue(c, case, st["residual"])
    if op == "mx":
        c = _exact_mx(st["x"], st["sx"]) @ _exact_mx(st["B"], st["sB"]).t().contiguous()
        if st["bias"] is not None:
            c = c + st["bias"].double()
        y = _exact_epilogue(c, case, st["residual"])
    else:
        M, W = st["x"].shape[0], st["B"].shape[1]
        c = torch.zeros(M, W, dtype=torch.float64, device=DEV)
        for e, (a, b) in enumerate(zip(ends, ends[1:])):
            if a == b:
                continue
            if op == "i8_experts":
                x = st["x"][a:b].double() * st["sx"][a:b].double()[:, None]
                w = st["B"][e].double() * st["sB"][e].double()[:, None]
            else:
                x, w = _exact_mx(st["x"][a:b], st["sx"][a:b]), _exact_mx(st["B"][e], st["sB"][e])
            c[a:b] = x @ w.t().contiguous()
            if st["bias"] is not None:
                c[a:b] += st["bias"][e].double()
        y = _exact_epilogue(c, case, None)
        if op == "i8_experts":
            return y
    return {"y": y, "pre": c} if case["keep"] else {"y": y}
