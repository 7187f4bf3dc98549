"""GPU tests of the routed-expert operators against plain numpy forms in
binary64 (routed_oracle).

Tolerances, derived from the operations (u = 2^-24, half an ulp of fp32):
  * a probability: the score's difference from the row's largest rounds once
    (|d| u), its product with log2 e twice more (2 |d| u), exp2 and the
    division and product are within 4 ulp together (8 u), the row's sum of E
    terms adds E u at most; the sum's own terms carry 3 D u for the row's
    largest |d| = D.  Renormalized weights do this twice:
        |w - w64| <= w (6 D + 2 E + 32) u, and 2^-120 where exp underflows.
  * prob: T terms more, (T + 6 D + 2 E + 32) u; loss: E more.
  * dlogits: products and a sum of E terms of the above,
        (12 D + 6 E + 64) u of the magnitudes that went in; T u of the loss's
    part through counts / live is exact in the oracle's inputs.  bf16 results
    round once more, 2^-8 |d|.
  * codes, scales, copies, gradient rows: equal bits (each operation is one
    fp32 rounding of the same operands).
  * products: the integer sum is exact; its conversion, two products and the
    bias add round once each: 4 u of the magnitudes, then the output's own
    2^-8 |C| in bf16.
  * combine: k fused multiply-adds, k u of the magnitudes, then 2^-8 |y|.
  * dweight: a thread adds N/256 + 16 terms in turn at most, then 8 levels.
"""
import numpy as np
import pytest
import torch

import mx9_dual_axis_amd as mxq
import routed_oracle as ro
from helpers import require_gpu, say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = ro.U
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _gpu(request):
    require_gpu()
    say(request.node.name)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def ints(t):
    return t.cpu().numpy()


def pitched(a, dtype, pitch_extra=0, offset=0):
    """a (numpy) on the device with rows `pitch_extra` elements apart from
    contiguous and the base `offset` elements past an aligned one."""
    rows, cols = a.shape
    buf = torch.full((offset + rows * (cols + pitch_extra) + 8,), 77, dtype=dtype, device=DEV)
    v = buf[offset:].as_strided((rows, cols), (cols + pitch_extra, 1))
    v.copy_(torch.from_numpy(np.ascontiguousarray(a)).to(dtype))
    return v


def close(got, want, tol, what):
    bad = ~(np.abs(got - want) <= tol) & ~(np.isnan(got) & np.isnan(want))
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        pytest.fail(f"{what}: {bad.sum()} of {bad.size} beyond the bound; first {i}: got {got[i]!r} want {want[i]!r} "
                    f"tol {np.broadcast_to(tol, got.shape)[i]!r}")


# -------------------------------------------------------------------- routing
def make_logits(T, E, seed, dtype, barred=0.05, coarse=False):
    g = np.random.default_rng(seed)
    z = g.normal(size=(T, E)) * 2 + g.normal(size=E)
    if coarse:                                      # many equal scores, zeros of both signs among them
        z = np.round(z)
        z[g.random((T, E)) < 0.1] = -0.0
    z[g.random((T, E)) < barred] = -np.inf
    return torch.from_numpy(z).to(DT[dtype])


def check_route(z, valid, k, normalize, align, r, tag):
    zz = z.double().numpy()
    T, E = zz.shape
    w = ro.route(zz, valid, k, normalize, align, r.rows)
    for n in ("idx", "slot", "src", "counts", "offs"):
        got = ints(getattr(r, n))
        assert np.array_equal(got, w[n]), f"{tag}: {n} differs at {np.argwhere(got != w[n])[:3].tolist()}"
    assert int(r.live) == w["live"], tag
    D = ro.route_spread(zz)
    e = (6 * D + 2 * E + 32) * U
    close(f64(r.weight), w["weight"], w["weight"] * e + 2.0 ** -120, f"{tag}: weight")
    close(f64(r.prob), w["prob"], w["prob"] * (e + T * U) + 2.0 ** -120, f"{tag}: prob")
    close(f64(r.loss), np.array([w["loss"]]), np.array([abs(w["loss"]) * (e + (T + E) * U) + 2.0 ** -120]), f"{tag}: loss")
    return w, D


def check_grad(z, valid, w, D, r, normalize, dw, dl, got, tag, dtype):
    T, E = z.shape
    d, mag = ro.route_grad(z.double().numpy(), w, r.k, normalize, dw.astype(np.float64), float(dl))
    tol = mag * (12 * D + 6 * E + 64) * U + 2.0 ** -120
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * np.abs(d)
    if valid is not None:
        d[~valid] = 0
    close(f64(got), d, tol, f"{tag}: dlogits")


ROUTE = [
    # T, E, k, align, dtype
    (1, 1, 1, 1, "f32"), (1, 64, 4, 1, "bf16"), (2, 5, 5, 16, "f32"), (63, 16, 16, 3, "bf16"), (64, 17, 2, 128, "f32"),
    (65, 60, 8, 128, "bf16"), (129, 64, 8, 1, "f32"), (500, 160, 6, 7, "bf16"), (300, 256, 8, 128, "f32"),
    (97, 300, 9, 1, "bf16"), (70, 513, 16, 2, "f32"), (40, 1024, 16, 1, "bf16"), (1031, 1024, 1, 1, "f32"),
    (5000, 33, 3, 128, "f32"),
]


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,E,k,align,dtype", ROUTE)
def test_route_and_gradient(T, E, k, align, dtype, normalize):
    g = np.random.default_rng(T * 7 + E)
    z = make_logits(T, E, T + E, dtype)
    valid = g.random(T) < 0.9
    zd = z.clone()
    zd[~torch.from_numpy(valid)] = float("nan")      # what is masked may hold anything
    zd = zd.to(DEV)
    vd = torch.from_numpy(valid).to(DEV)
    r = mxq.mx_route(zd, k, valid=vd, normalize=normalize, align=align)
    w, D = check_route(z, valid, k, normalize, align, r, f"T={T} E={E}")
    dw = g.normal(size=(T, k)).astype(np.float32)
    dl = np.float32(0.37)
    got = mxq.mx_route_grad(zd, r, torch.from_numpy(dw).to(DEV), torch.full((1,), float(dl), device=DEV), valid=vd)
    assert got.dtype == DT[dtype]
    check_grad(z, valid, w, D, r, normalize, dw, dl, got, f"T={T} E={E}", dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,k", [(50, 24, 6), (700, 128, 8)])
def test_route_equal_scores_go_to_the_lowest_expert(T, E, k, dtype):
    z = make_logits(T, E, 3, dtype, coarse=True)
    r = mxq.mx_route(z.to(DEV), k, align=4)
    check_route(z, None, k, True, 4, r, "ties")


@pytest.mark.parametrize("T", [20, 200])
def test_route_rows_with_little_or_nothing_left(T):
    E, k = 12, 4
    z = make_logits(T, E, 9, "f32", barred=0)
    z[3] = -np.inf                                   # nothing
    z[4, 1:] = -np.inf                               # one expert
    z[5, [0, 2, 3, 5, 6, 7, 8, 9, 10]] = -np.inf     # fewer than k
    z[6] = torch.finfo(torch.float32).min            # the type's lowest value is a score like any other
    z[7, :6] = torch.finfo(torch.float32).min
    for normalize in (True, False):
        r = mxq.mx_route(z.to(DEV), k, normalize=normalize, align=8)
        zz = z.double().numpy()
        w = ro.route(zz, None, k, normalize, 8, r.rows)
        for n in ("idx", "slot", "src", "counts", "offs"):
            assert np.array_equal(ints(getattr(r, n)), w[n]), n
        fin = z.clone()
        fin[7, :6] = -np.inf                         # their probability is 0 in any precision
        close(f64(r.weight), w["weight"], w["weight"] * (6 * 20 + 2 * E + 32) * U + 2.0 ** -120, "weight")
        d = mxq.mx_route_grad(z.to(DEV), r, torch.ones(T, k, device=DEV), torch.ones(1, device=DEV))
        d = f64(d)
        assert np.isfinite(d).all()
        assert (d[3] == 0).all() and (d[z.numpy() == -np.inf] == 0).all()


@pytest.mark.parametrize("T", [8, 130])
def test_route_with_no_live_token(T):
    z = torch.full((T, 6), float("-inf"), device=DEV)
    z2 = torch.full((T, 6), float("nan"), device=DEV)
    none = torch.zeros(T, dtype=torch.uint8, device=DEV)
    for zz, v in ((z, None), (z2, none)):
        r = mxq.mx_route(zz, 3, valid=v, align=4)
        assert (ints(r.idx) == -1).all() and (ints(r.slot) == -1).all() and (ints(r.src) == -1).all()
        assert not ints(r.counts).any() and not ints(r.offs).any() and int(r.live) == 0
        assert not f64(r.weight).any() and not f64(r.prob).any() and float(r.loss) == 0
        d = mxq.mx_route_grad(zz, r, torch.ones(T, 3, device=DEV), torch.ones(1, device=DEV), valid=v)
        assert not f64(d).any()


def test_route_of_no_tokens():
    r = mxq.mx_route(torch.empty((0, 6), device=DEV), 3, align=4)
    assert r.rows == 0 and not ints(r.counts).any() and not ints(r.offs).any() and int(r.live) == 0 and float(r.loss) == 0
    assert mxq.mx_route_grad(torch.empty((0, 6), device=DEV), r).shape == (0, 6)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("T", [30, 300])
def test_route_with_a_bad_score(T, bad):
    E, k = 20, 3
    z = make_logits(T, E, 4, "f32")
    z[11, 7] = bad
    r = mxq.mx_route(z.to(DEV), k, align=2)
    w = ro.route(z.double().numpy(), None, k, True, 2, r.rows)
    for n in ("idx", "slot", "src", "counts", "offs"):
        assert np.array_equal(ints(getattr(r, n)), w[n]), n
    assert int(r.live) == w["live"]
    wt = f64(r.weight)
    assert np.isnan(wt[11]).all() and np.isfinite(np.delete(wt, 11, 0)).all()
    assert np.isnan(f64(r.prob)).all() and np.isnan(float(r.loss))
    d = f64(mxq.mx_route_grad(z.to(DEV), r, torch.ones(T, k, device=DEV)))
    assert np.isnan(d[11]).all() and np.isfinite(np.delete(d, 11, 0)).all()


@pytest.mark.parametrize("dtype,extra,offset", [("bf16", 3, 1), ("f32", 5, 3), ("bf16", 8, 0)])
def test_route_pitched_logits(dtype, extra, offset):
    T, E, k = 150, 40, 4
    z = make_logits(T, E, 8, dtype)
    zd = pitched(z.float().numpy(), DT[dtype], extra, offset)
    r = mxq.mx_route(zd, k, align=16)
    w, D = check_route(z, None, k, True, 16, r, "pitched")
    dw = np.random.default_rng(1).normal(size=(T, k)).astype(np.float32)
    buf = torch.full((T, E + 5), 55, dtype=DT[dtype], device=DEV)
    got = mxq.mx_route_grad(zd, r, torch.from_numpy(dw).to(DEV), out=buf[:, :E])
    check_grad(z, None, w, D, r, True, dw, 0.0, got, "pitched", dtype)
    assert (buf[:, E:] == 55).all()


@pytest.mark.parametrize("normalize", [True, False])
def test_route_gradient_against_differences(normalize):
    """The kernel's gradient against differences of its own forward in fp32:
    step 2^-5, so the third-order term is below 2^-10 of the terms and the
    forward's rounding, 2^-21 over 2^-4, below 2^-16."""
    T, E, k = 12, 10, 3
    g = np.random.default_rng(2)
    z = torch.from_numpy(np.stack([g.permutation(E) for _ in range(T)]) * 0.5).float()   # gaps of 0.5: picks hold
    dw = torch.from_numpy(g.normal(size=(T, k))).float()

    def f(zz):
        r = mxq.mx_route(zz.to(DEV), k, normalize=normalize)
        return (f64(r.weight) * dw.double().numpy()).sum(1), float(r.loss)

    r = mxq.mx_route(z.to(DEV), k, normalize=normalize)
    d = f64(mxq.mx_route_grad(z.to(DEV), r, dw.to(DEV)))
    dl = f64(mxq.mx_route_grad(z.to(DEV), r, dloss=torch.ones(1, device=DEV)))
    h = 2.0 ** -5
    for e in range(E):
        a, b = z.clone(), z.clone()
        a[:, e] += h
        b[:, e] -= h
        close((f(a)[0] - f(b)[0]) / (2 * h), d[:, e], 2.0 ** -9 * np.abs(dw.numpy()).sum(1), f"weights by score {e}")
        for t in (0, 5):
            a, b = z.clone(), z.clone()
            a[t, e] += h
            b[t, e] -= h
            num = (f(a)[1] - f(b)[1]) / (2 * h)
            assert abs(num - dl[t, e]) < 2.0 ** -9 * E / T + 2.0 ** -16, (t, e, num, dl[t, e])


def test_route_repeats_bit_for_bit():
    z = make_logits(3000, 96, 6, "bf16").to(DEV)
    dw = torch.randn(3000, 6, device=DEV)
    a = mxq.mx_route(z, 6)
    da = mxq.mx_route_grad(z, a, dw, torch.ones(1, device=DEV))
    for _ in range(3):
        b = mxq.mx_route(z, 6)
        for n in ("idx", "weight", "slot", "src", "counts", "offs", "live", "prob", "loss"):
            assert torch.equal(getattr(a, n), getattr(b, n)), n
        assert torch.equal(da, mxq.mx_route_grad(z, b, dw, torch.ones(1, device=DEV)))


def test_route_out_is_reused_and_checked():
    plan = mxq.mx_routing(100, 32, 4, align=8, device=DEV)
    for seed in (1, 2):
        z = make_logits(100, 32, seed, "f32")
        assert mxq.mx_route(z.to(DEV), 4, out=plan) is plan
        check_route(z, None, 4, True, 8, plan, "reused")
    for z, k in ((torch.zeros(99, 32, device=DEV), 4), (torch.zeros(100, 31, device=DEV), 4), (torch.zeros(100, 32, device=DEV), 3)):
        with pytest.raises(ValueError):
            mxq.mx_route(z, k, out=plan)
    with pytest.raises(ValueError):
        mxq.mx_route(torch.zeros(100, 32, device=DEV, dtype=torch.float16), 4)
    with pytest.raises(ValueError):
        mxq.mx_route(torch.zeros(100, 32, device=DEV), 4, valid=torch.ones(99, dtype=torch.bool, device=DEV))
    with pytest.raises(ValueError):
        mxq.mx_route_grad(torch.zeros(100, 32, device=DEV), plan, torch.ones(100, 3, device=DEV))


# ------------------------------------------------- dispatch, quantized or not
def make_map(T, k, E, align, seed, drop=0.1):
    """A row map as routing makes it: (slot, src, offs, M) in numpy."""
    g = np.random.default_rng(seed)
    groups = [[] for _ in range(E)]
    slot = np.full((T, k), -1, np.int32)
    for t in range(T):
        for j, e in enumerate(g.permutation(E)[:k]):
            if g.random() >= drop:
                groups[e].append((t, j))
    M = ro.rows_needed(T, E, k, align)
    src, offs, at = np.full(M, -1, np.int32), np.zeros(E, np.int32), 0
    for e in range(E):
        for r, (t, j) in enumerate(groups[e]):
            slot[t, j] = at + r
            src[at + r] = t * k + j
        at += -(-len(groups[e]) // align) * align
        offs[e] = at
    return slot, src, offs, M


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


SHAPES = [(1, 1, 1, 1, 1), (5, 1, 3, 2, 4), (3, 7, 4, 2, 1), (9, 8, 3, 3, 2), (17, 9, 5, 2, 16), (33, 64, 8, 4, 1),
          (64, 511, 16, 8, 128), (37, 1111, 10, 3, 1), (20, 2049, 6, 2, 3), (6, 9001, 3, 2, 2)]
# T, N, E, k, align


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,E,k,align", SHAPES)
@pytest.mark.parametrize("extra,offset", [(0, 0), (3, 1)])
def test_dispatch(T, N, E, k, align, dtype, extra, offset):
    slot, src, offs, M = make_map(T, k, E, align, T + N)
    x = pitched(np.random.default_rng(N).normal(size=(T, N)), DT[dtype], extra, offset)
    buf = torch.full((M, N + extra), 99, dtype=DT[dtype], device=DEV)
    out = mxq.mx_dispatch(x, dev(slot), dev(src), out=buf[:, :N])
    want = torch.zeros(M, N, dtype=DT[dtype])
    for t in range(T):
        for j in range(k):
            if slot[t, j] >= 0:
                want[slot[t, j]] = x[t].cpu()
    assert torch.equal(out.cpu(), want)
    assert (buf[:, N:] == 99).all()
    if extra == 0:
        assert torch.equal(mxq.mx_dispatch(x, dev(slot), dev(src)).cpu(), want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,E,k,align", SHAPES)
@pytest.mark.parametrize("extra,offset", [(0, 0), (3, 1)])
def test_quantized_rows(T, N, E, k, align, dtype, extra, offset):
    slot, src, offs, M = make_map(T, k, E, align, T + N)
    g = np.random.default_rng(N)
    a = g.normal(size=(T, N)) * np.exp(3 * g.normal(size=(T, 1)))
    x = pitched(a, DT[dtype], extra, offset)
    wq, ws = ro.quantize(x.float().cpu().numpy())
    q, s = mxq.i8_quantize_rows(x)
    assert np.array_equal(ints(q), wq) and np.array_equal(ints(s), ws)
    buf = torch.full((M, N + extra), 99, dtype=torch.int8, device=DEV)
    qd, sd = mxq.mx_dispatch_i8(x, dev(slot), dev(src), out=(buf[:, :N], torch.empty(M, device=DEV)))
    full_q, full_s = np.zeros((M, N), np.int8), np.full(M, np.float32(2.0 ** -126), np.float32)
    for t in range(T):
        for j in range(k):
            if slot[t, j] >= 0:
                full_q[slot[t, j]], full_s[slot[t, j]] = wq[t], ws[t]
    assert np.array_equal(ints(qd), full_q) and np.array_equal(ints(sd), full_s)
    assert (buf[:, N:] == 99).all()
    if extra == 0:
        qd, sd = mxq.mx_dispatch_i8(x, dev(slot), dev(src))
        assert np.array_equal(ints(qd), full_q) and np.array_equal(ints(sd), full_s)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [1, 5, 40, 5000, 17000])
def test_quantized_special_rows(K, dtype):
    big = 3.3e38
    a = np.random.default_rng(3).normal(size=(10, K)).astype(np.float32)
    a[0] = 0
    a[1] = -0.0
    a[2] = 0
    a[2, K // 2] = 2.0 ** -149 if dtype == "f32" else 2.0 ** -133       # a lone subnormal
    a[3] *= np.float32(2.0 ** -130)                                      # a row of subnormals
    a[4, K - 1] = np.inf
    a[5, 0] = np.nan
    a[6, K // 2] = -np.inf
    a[7] = np.sign(a[7]) * big
    a[8, 0] = 1e-30
    a[9] = np.linspace(-1, 1, K) if K > 1 else 1
    x = torch.from_numpy(a).to(DT[dtype]).to(DEV)
    wq, ws = ro.quantize(x.float().cpu().numpy())
    q, s = mxq.i8_quantize_rows(x)
    assert np.array_equal(ints(q), wq)
    assert np.array_equal(ints(s), ws, equal_nan=True)
    # what comes of a bad row is NaN, and of no other
    B, sB = torch.ones((3, K), dtype=torch.int8, device=DEV), torch.ones(3, device=DEV)
    c = f64(mxq.i8_linear(x, B, sB, out_dtype=torch.float32))
    assert np.isnan(c[[4, 5, 6]]).all() and not np.isnan(np.delete(c, [4, 5, 6], 0)).any()


def test_row_maps_that_point_outside_are_skipped():
    T, N, k, M = 6, 40, 2, 12
    slot = np.arange(T * k, dtype=np.int32).reshape(T, k)
    slot[1, 0], slot[2, 1], slot[3, 0] = M, 2 ** 31 - 1, -7
    src = np.where(np.isin(np.arange(M), slot), np.arange(M), -1).astype(np.int32)
    x = torch.randn(T, N, device=DEV)
    want = np.zeros((M, N))
    for t in range(T):
        for j in range(k):
            if 0 <= slot[t, j] < M:
                want[slot[t, j]] = f64(x)[t]
    assert np.array_equal(f64(mxq.mx_dispatch(x, dev(slot), dev(src))), want)
    rows = torch.randn(M, N, device=DEV)
    y, mag = ro.combine(f64(rows), slot, None)
    close(f64(mxq.mx_combine(rows, dev(slot))), y, k * U * mag, "combine")
    q, s = mxq.mx_dispatch_i8(x, dev(slot), dev(src))
    assert (ints(q)[want.any(1)] != 0).any() and not ints(q)[~want.any(1)].any()
    d, dw = mxq.mx_combine_grad(x, rows, dev(slot), None, dev(src))
    assert np.array_equal(f64(d), want) and f64(dw)[1, 0] == 0 and f64(dw)[2, 1] == 0 and f64(dw)[3, 0] == 0


# -------------------------------------------------------------------- combine
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,E,k,align", SHAPES)
@pytest.mark.parametrize("extra,offset", [(0, 0), (3, 1)])
def test_combine_and_gradient(T, N, E, k, align, dtype, extra, offset):
    slot, src, offs, M = make_map(T, k, E, align, T + N, drop=0.3)
    g = np.random.default_rng(N + 1)
    rows = pitched(g.normal(size=(M, N)), DT[dtype], extra, offset)
    dy = pitched(g.normal(size=(T, N)), DT[dtype], extra, offset)
    w = g.normal(size=(T, k)).astype(np.float32)
    w[slot < 0] = np.nan                              # what has no slot takes no part
    R, G = f64(rows), f64(dy)
    for weight in (None, w):
        wd = None if weight is None else dev(weight)
        y, mag = ro.combine(R, slot, weight)
        tol = k * U * mag + (2.0 ** -8 * np.abs(y) if dtype == "bf16" else 0)
        buf = torch.full((T, N + extra), 99, dtype=DT[dtype], device=DEV)
        close(f64(mxq.mx_combine(rows, dev(slot), wd, out=buf[:, :N])), y, tol, "y")
        assert (buf[:, N:] == 99).all()
        dbuf = torch.full((M, N + extra), 99, dtype=DT[dtype], device=DEV)
        dw = torch.full((T, k), 5.0, device=DEV)
        mxq.mx_combine_grad(dy, rows, dev(slot), wd, dev(src), out=(dbuf[:, :N], dw))
        assert (dbuf[:, N:] == 99).all()
        want = torch.zeros(M, N, dtype=DT[dtype])
        wdot, dmag = np.zeros((T, k)), np.zeros((T, k))
        for t in range(T):
            for j in range(k):
                r = slot[t, j]
                if r >= 0:
                    f = 1.0 if weight is None else weight[t, j]
                    want[r] = (torch.tensor(f, dtype=torch.float32) * dy[t].cpu().float()).to(DT[dtype])
                    wdot[t, j] = G[t] @ R[r]
                    dmag[t, j] = np.abs(G[t]) @ np.abs(R[r])
        assert torch.equal(dbuf[:, :N].cpu(), want)
        close(f64(dw), wdot, (N / 256 + 16 + 8) * U * dmag, "dweight")


def test_combine_gradient_against_differences():
    """combine is linear in the rows and in the weights: differences at any
    step give its gradient up to the rounding of the two sums."""
    T, N, E, k = 7, 24, 5, 2
    slot, src, offs, M = make_map(T, k, E, 2, 3, drop=0.2)
    g = np.random.default_rng(8)
    rows, dy = torch.from_numpy(g.normal(size=(M, N))).float().to(DEV), g.normal(size=(T, N))
    w = torch.from_numpy(g.normal(size=(T, k))).float().to(DEV)
    dyt = torch.from_numpy(dy).float().to(DEV)
    d, dw = mxq.mx_combine_grad(dyt, rows, dev(slot), w, dev(src))

    def f(rows, w):
        return float((f64(mxq.mx_combine(rows, dev(slot), w)) * f64(dyt)).sum())

    for r in range(M):
        a, b = rows.clone(), rows.clone()
        a[r, r % N] += 1
        b[r, r % N] -= 1
        assert abs((f(a, w) - f(b, w)) / 2 - f64(d)[r, r % N]) < 1e-4
    for t in range(T):
        a, b = w.clone(), w.clone()
        a[t, t % k] += 1
        b[t, t % k] -= 1
        assert abs((f(rows, a) - f(rows, b)) / 2 - f64(dw)[t, t % k]) < 1e-4


def test_dispatch_then_combine_is_its_own_gradient():
    """<dispatch(x), R> = <x, combine(R)> with every weight 1 (integers: exact)."""
    T, N, E, k = 50, 96, 8, 3
    slot, src, offs, M = make_map(T, k, E, 4, 1)
    g = np.random.default_rng(0)
    x, R = dev(g.integers(-4, 5, (T, N)).astype(np.float32)), dev(g.integers(-4, 5, (M, N)).astype(np.float32))
    a = (mxq.mx_dispatch(x, dev(slot), dev(src)).double() * R.double()).sum()
    b = (x.double() * mxq.mx_combine(R, dev(slot)).double()).sum()
    assert float(a) == float(b)


# ------------------------------------------------------------------- products
def codes(g, shape, full=False):
    return g.integers(-128 if full else -127, 128, shape, dtype=np.int64).astype(np.int8)


PRODUCTS = [
    # M, N, K
    (1, 1, 1), (1, 1, 0), (1, 37, 15), (2, 16, 16), (1, 300, 17), (3, 130, 63), (16, 64, 64), (17, 129, 65), (31, 40, 127),
    (32, 256, 128), (33, 100, 129), (64, 96, 1000), (65, 513, 257), (100, 31, 4097), (128, 128, 512), (130, 257, 384),
    (200, 1000, 1111), (256, 256, 1024), (257, 511, 640), (384, 768, 2048), (1, 4096, 4096), (8, 2048, 5120),
    (513, 300, 72), (1000, 520, 48),
]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product(M, N, K, out):
    g = np.random.default_rng(M + N + K)
    a, b = codes(g, (M, K)), codes(g, (N, K))
    sa, sb = np.exp(g.normal(size=M)).astype(np.float32), np.exp(g.normal(size=N)).astype(np.float32)
    bias = (g.normal(size=N) * 50).astype(np.float32)
    for extra, offset, bi in ((0, 0, None), (16, 0, bias), (5, 3, bias)):
        A, B = pitched(a, torch.int8, extra, offset), pitched(b, torch.int8, extra, offset)
        want, mag = ro.product(a, sa, b, sb, bi)
        tol = 4 * U * mag + (2.0 ** -8 * np.abs(want) if out == "bf16" else 0)
        buf = torch.full((M, N + extra), 99, dtype=DT[out], device=DEV)
        got = mxq.i8_gemm_nt(A, dev(sa), B, dev(sb), None if bi is None else dev(bi), out=buf[:, :N])
        close(f64(got), want, tol, f"pitch +{extra}, base +{offset}")
        assert (buf[:, N:] == 99).all()


@pytest.mark.parametrize("M,N,K", [(1, 64, 64), (5, 33, 200), (40, 200, 700), (128, 256, 640), (300, 300, 1000)])
def test_product_is_exact_in_integers(M, N, K):
    """Unit scales and sums below 2^24: the fp32 result is the integer."""
    g = np.random.default_rng(K)
    a, b = codes(g, (M, K), full=True), codes(g, (N, K), full=True)
    one = lambda n: torch.ones(n, device=DEV)  # noqa: E731
    got = mxq.i8_gemm_nt(dev(a), one(M), dev(b), one(N), out_dtype=torch.float32)
    assert np.array_equal(f64(got), a.astype(np.int64) @ b.astype(np.int64).T)


@pytest.mark.parametrize("M", [1, 20, 130])
def test_product_of_the_largest_sums(M):
    """-128 times -128 over the longest contraction, 131071 * 2^14, just fits
    the 32-bit sum; fp32 holds 131071 * 2^14 exactly (17 bits)."""
    K, N = 131071, 130
    A = torch.full((M, K), -128, dtype=torch.int8, device=DEV)
    B = torch.full((N, K), -128, dtype=torch.int8, device=DEV)
    got = mxq.i8_gemm_nt(A, torch.ones(M, device=DEV), B, torch.ones(N, device=DEV), out_dtype=torch.float32)
    assert (got == 131071.0 * 16384.0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 40, 100), (1, 2048, 4096), (2, 300, 9001), (7, 130, 513), (16, 64, 64), (77, 1000, 1111),
                                   (130, 260, 640), (300, 100, 31)])
def test_linear(M, N, K, dtype):
    g = np.random.default_rng(M * N)
    x = pitched(g.normal(size=(M, K)) * np.exp(g.normal(size=(M, 1))), DT[dtype], 3 if K == 513 else 0, 0)
    b, sb = codes(g, (N, K)), np.exp(g.normal(size=N)).astype(np.float32)
    bias = g.normal(size=N).astype(np.float32)
    qa, sa = ro.quantize(x.float().cpu().numpy())
    for bi in (None, bias):
        want, mag = ro.product(qa, sa, b, sb, bi)
        for out in ("f32", "bf16"):
            tol = 4 * U * mag + (2.0 ** -8 * np.abs(want) if out == "bf16" else 0)
            got = mxq.i8_linear(x, dev(b), dev(sb), None if bi is None else dev(bi), out_dtype=DT[out])
            close(f64(got), want, tol, f"{out}")
    assert mxq.i8_linear(x, dev(b), dev(sb)).dtype == DT[dtype]


def check_grouped(sizes, tail, N, K, seed, out="bf16", offs=None, extra=0, offset=0):
    g = np.random.default_rng(seed)
    offs = np.cumsum(sizes).astype(np.int32) if offs is None else np.array(offs, np.int32)
    M, G = int(sum(sizes) + tail), len(offs)
    a, b = codes(g, (M, K)), codes(g, (G, N, K))
    sa, sb = np.exp(g.normal(size=M)).astype(np.float32), np.exp(g.normal(size=(G, N))).astype(np.float32)
    sa[max(0, ro.group_ranges(offs, M)[-1][1]):] = np.nan    # the tail belongs to nobody, whatever it holds
    A = pitched(a, torch.int8, extra, offset)
    B = pitched(b.reshape(G * N, K), torch.int8, extra, offset).unflatten(0, (G, N)) if extra or offset else dev(b)
    got = f64(mxq.i8_grouped_gemm_rows(A, dev(sa), B, dev(sb), dev(offs), out_dtype=DT[out]))
    want, mag = np.zeros((M, N)), np.zeros((M, N))
    for e, (r0, r1) in enumerate(ro.group_ranges(offs, M)):
        want[r0:r1], mag[r0:r1] = ro.product(a[r0:r1], np.nan_to_num(sa[r0:r1]), b[e], sb[e])
    close(got, want, 4 * U * mag + (2.0 ** -8 * np.abs(want) if out == "bf16" else 0), f"sizes {list(sizes)[:8]}")


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("sizes,tail,N,K", [
    ([1], 0, 16, 16), ([0, 0, 3], 0, 40, 64), ([0, 0], 5, 33, 100), ([1, 2, 0, 5, 16, 17], 3, 130, 128),
    ([128, 256, 0, 128], 128, 256, 256), ([100, 300, 1, 129], 77, 300, 640), ([3] * 70, 9, 64, 192),
    ([0] * 130 + [4, 5], 2, 48, 65), ([512, 384], 0, 512, 1024), ([40, 90, 33, 64], 1, 200, 513),
    ([700, 3, 0, 400], 10, 136, 48)])
def test_grouped_product(sizes, tail, N, K, out):
    check_grouped(sizes, tail, N, K, sum(sizes) + N, out)
    check_grouped(sizes, tail, N, K, sum(sizes) + N, out, extra=16)
    check_grouped(sizes, tail, N, K, sum(sizes) + N, out, extra=5, offset=3)


@pytest.mark.parametrize("seed", range(6))
def test_grouped_product_random_sizes(seed):
    g = np.random.default_rng(seed)
    G = int(g.integers(1, 90))
    sizes = (g.integers(0, 60, G) * (g.random(G) < 0.7)).tolist()
    check_grouped(sizes, int(g.integers(0, 200)), int(g.integers(1, 400)), int(g.integers(1, 700)), seed)


@pytest.mark.parametrize("offs", [[50, 20, 200, 90], [-5, 30, 30, 1000], [2 ** 31 - 1, 0, 0, 0], [-1, -2, -3, -2 ** 31]])
def test_grouped_product_with_invalid_offsets(offs):
    """Clamped to an ascending sequence within the rows, as the header says."""
    check_grouped([100, 100], 40, 70, 96, 5, offs=offs)


# ------------------------------------------- big operands, streams and graphs
def test_offsets_past_32_bits():
    """Rows, codes and results beyond 2^31 bytes and elements."""
    N, T, M = 32768, 8, 70000
    slot = torch.tensor([[i] for i in (0, 1, 40000, 65535, 65536, 65537, 69998, 69999)], dtype=torch.int32, device=DEV)
    src = torch.full((M,), -1, dtype=torch.int32, device=DEV)
    src[slot[:, 0].long()] = torch.arange(T, dtype=torch.int32, device=DEV)
    x = torch.randn(T, N, device=DEV).to(torch.bfloat16)
    rows = mxq.mx_dispatch(x, slot, src)
    assert torch.equal(rows[slot[:, 0].long()], x) and int((rows != 0).any(1).sum()) == T
    assert torch.equal(mxq.mx_combine(rows, slot), x)
    q, s = mxq.mx_dispatch_i8(x, slot, src)
    w, sw = mxq.i8_quantize_rows(torch.randn(5, N, device=DEV))
    small = mxq.i8_gemm_nt(q[slot[:, 0].long()].contiguous(), s[slot[:, 0].long()].contiguous(), w, sw)
    assert torch.equal(mxq.i8_gemm_nt(q, s, w, sw)[slot[:, 0].long()], small)
    del rows, q, s
    # the last of many experts, each 64 MiB of codes
    G, N, K = 40, 8192, 8192
    B = torch.zeros((G, N, K), dtype=torch.int8, device=DEV)
    B[G - 1] = torch.randint(-127, 128, (N, K), dtype=torch.int8, device=DEV)
    sB = torch.ones((G, N), device=DEV)
    A, sA = torch.randint(-127, 128, (9, K), dtype=torch.int8, device=DEV), torch.ones(9, device=DEV)
    offs = torch.full((G,), 4, dtype=torch.int32, device=DEV)
    offs[G - 1] = 9
    c = mxq.i8_grouped_gemm_rows(A, sA, B, sB, offs)
    assert not c[:4].any() and torch.equal(c[4:], mxq.i8_gemm_nt(A[4:], sA[4:], B[G - 1], sB[G - 1]))
    del B
    # a result of more than 2^31 elements
    M, N = 70000, 32000
    A, sA = torch.zeros((M, 16), dtype=torch.int8, device=DEV), torch.ones(M, device=DEV)
    A[M - 3:] = 2
    Bw, sw = torch.ones((N, 16), dtype=torch.int8, device=DEV), torch.ones(N, device=DEV)
    c = mxq.i8_gemm_nt(A, sA, Bw, sw)
    assert (c[M - 3:] == 32).all() and not c[:M - 3].any()


def layer(x, z, W1, s1, W2, s2, k, plan):
    mxq.mx_route(z, k, out=plan)
    q, s = mxq.mx_dispatch_i8(x, plan.slot, plan.src)
    h = mxq.i8_grouped_gemm_rows(q, s, W1, s1, plan.offs)
    q2, s2_ = mxq.i8_quantize_rows(torch.relu(h))
    o = mxq.i8_grouped_gemm_rows(q2, s2_, W2, s2, plan.offs)
    return mxq.mx_combine(o, plan.slot, plan.weight)


def make_layer(T, seed=0):
    E, k, K, H = 8, 2, 256, 320
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn(T, K, generator=g, device=DEV).to(torch.bfloat16)
    z = torch.randn(T, E, generator=g, device=DEV)
    W1, s1 = mxq.i8_quantize_rows(torch.randn(E * H, K, generator=g, device=DEV))
    W2, s2 = mxq.i8_quantize_rows(torch.randn(E * K, H, generator=g, device=DEV))
    return [x, z, W1.view(E, H, K), s1.view(E, H), W2.view(E, K, H), s2.view(E, K), k,
            mxq.mx_routing(T, E, k, align=1, device=DEV)]


@pytest.mark.parametrize("T", [3, 100])
def test_layer_in_a_graph(T):
    a = make_layer(T)
    want = layer(*a).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(*a)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(*a)
    x0, z0 = a[0].clone(), a[1].clone()
    for i in range(4):
        b = make_layer(T, seed=i + 1)
        a[0].copy_(b[0])
        a[1].copy_(b[1])
        graph.replay()
        torch.cuda.synchronize()
        eager = layer(b[0], b[1], *a[2:7], b[7])
        assert torch.equal(got, eager), i
    a[0].copy_(x0)
    a[1].copy_(z0)
    graph.replay()
    assert torch.equal(got, want)


def test_layers_on_two_streams_give_the_serial_results():
    a, b = make_layer(40, 1), make_layer(300, 2)
    want = [layer(*a).clone(), layer(*b).clone()]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s1):
            ya = layer(*a)
        with torch.cuda.stream(s2):
            yb = layer(*b)
        torch.cuda.synchronize()
        assert torch.equal(ya, want[0]) and torch.equal(yb, want[1])


def test_products_do_not_depend_on_the_batch():
    """A token's result has the same bits alone and in a batch of any size."""
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    x = torch.randn(400, 768, generator=g, device=DEV).to(torch.bfloat16)
    W, s = mxq.i8_quantize_rows(torch.randn(520, 768, generator=g, device=DEV))
    bias = torch.randn(520, generator=g, device=DEV)
    full = mxq.i8_linear(x, W, s, bias)
    for n in (1, 2, 5, 16, 17, 40, 100, 129, 257):
        assert torch.equal(mxq.i8_linear(x[:n], W, s, bias), full[:n]), n
