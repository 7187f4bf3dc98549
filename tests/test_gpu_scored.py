"""GPU tests of scored routing against binary64 (scored_oracle).

Picks, rows and counts are equal.  Weights: scored_oracle.weight_error.  prob
and loss: the shares' error, T additions of a batch (64 a block, then blocks)
and E of the loss.  Gradients: (12 D + 6 E + 6 k + 96) u of the magnitudes that
went in (scores once, sums of E and of k terms, divisions), 2^-8 of the result
in bf16.
"""
import numpy as np
import pytest
import torch

import mx9_dual_axis_amd as mxq
import scored_oracle as so
from helpers import require_gpu, say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = so.U


@pytest.fixture(autouse=True)
def _gpu(request):
    require_gpu()
    say(request.node.name)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def dev(a, dtype=torch.float32):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dtype).to(DEV)


def check(z, k, kind, bias=None, groups=1, top=None, best=2, normalize=True, scale=1.0, valid=None, align=1, out=None):
    """z: a device tensor.  Returns (routing, the binary64 one)."""
    T, E = z.shape
    top = groups if top is None else top
    got = mxq.mx_route_scored(z, k, bias=dev(bias), score=kind, groups=groups, top_groups=top, group_best=best,
                              normalize=normalize, scale=scale, valid=None if valid is None else dev(valid, torch.bool),
                              align=align, out=out)
    b = None if bias is None else bias.astype(np.float32).astype(np.float64)
    want = so.route(f64(z), k, kind, b, groups, top, best, normalize, scale, valid, align, got.rows)
    for n in ("idx", "counts", "offs", "slot", "src"):
        g = getattr(got, n).cpu().numpy()
        if not np.array_equal(g, want[n]):
            i = tuple(np.argwhere(g != want[n])[0])
            pytest.fail(f"{n}: {np.count_nonzero(g != want[n])} of {g.size} differ, first {i}: {g[i]}, want {want[n][i]}")
    assert int(got.live) == want["live"]
    w = f64(got.weight)
    err = so.weight_error(want, k, E, kind, normalize, scale)
    bad = ~(np.abs(w - want["weight"]) <= err) & ~(np.isnan(w) & np.isnan(want["weight"]))
    assert not bad.any(), (np.argwhere(bad)[0], w[bad][0], want["weight"][bad][0])
    if np.isnan(want["prob"]).any():
        assert got.prob.isnan().all() and got.loss.isnan().all()
    else:
        # a sigmoid score's e^-z is off by 1.25 |z| u, its argument being rounded once
        zs = np.abs(f64(z)[np.isfinite(f64(z))])
        one = (16 + 2 * zs.max(initial=0) + E + 24) * U if kind == "sigmoid" else (6 * want["spread"] + 2 * E + 32) * U
        e = one + (64 + T / 64 + 8) * U
        assert (np.abs(f64(got.prob) - want["prob"]) <= want["prob"] * e + 2.0 ** -118).all()
        assert abs(float(got.loss) - want["loss"]) <= want["loss"] * (e + (E + 8) * U) + 2.0 ** -118
    return got, want


def logits(T, E, dtype, g, spread=1.5):
    z = torch.from_numpy(g.standard_normal((T, E)) * spread).to(DT[dtype]).to(DEV)
    z[torch.from_numpy(g.random((T, E)) < 0.02).to(DEV)] = -torch.inf
    return z


# Every lane layout (E up to 16, 32, ... 1024, whole and ragged), one token to
# several blocks, groups of one expert to all of them.
@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,k,groups,top,best", [
    (1, 256, 8, 8, 4, 2), (4, 16, 4, 4, 2, 1), (5, 12, 12, 1, 1, 1), (64, 32, 6, 32, 9, 2), (65, 30, 5, 3, 1, 2),
    (130, 64, 8, 8, 3, 2), (777, 60, 6, 4, 2, 1), (300, 128, 16, 16, 2, 2), (200, 100, 4, 20, 6, 2), (2100, 256, 8, 8, 4, 2),
    (300, 160, 6, 8, 3, 1), (70, 512, 8, 16, 5, 2), (70, 400, 16, 25, 10, 1), (70, 1024, 16, 32, 7, 2), (70, 999, 8, 27, 4, 2),
    (66, 7, 1, 7, 1, 1), (66, 1, 1, 1, 1, 2), (66, 2, 2, 2, 2, 1)])
def test_by_size(T, E, k, groups, top, best, dtype, kind):
    g = np.random.default_rng(T + E)
    z = logits(T, E, dtype, g)
    bias = g.standard_normal(E) * 0.05
    check(z, k, kind, bias, groups, top, best, True, 2.5, align=4)
    check(z, k, kind, None, groups, top, best, False, 1.0, align=1)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
def test_pitches_alignments_and_plans(kind):
    g = np.random.default_rng(3)
    plan = mxq.mx_routing(150, 96, 5, align=16, device=DEV)
    for dtype in ("f32", "bf16"):
        z = logits(150, 96, dtype, g)
        wide = torch.full((150 * 103 + 9,), float("nan"), dtype=DT[dtype], device=DEV)
        v = wide[1:1 + 150 * 103].view(150, 103)[:, :96]
        v.copy_(z)
        r, _ = check(v, 5, kind, g.standard_normal(96) * 0.1, 6, 2, 2, align=16, out=plan)
        assert r is plan and plan.scored == (kind, 1.0)


# Tokens left out, rows that bar everything, a group or all but a few experts,
# NaN and infinite scores; biases that are not finite.
@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("biased", [False, True])
def test_masks(dtype, kind, biased):
    T, E, k = 200, 48, 6
    g = np.random.default_rng(5)
    z = torch.from_numpy(g.standard_normal((T, E)) * 2).to(DT[dtype])
    valid = g.random(T) < 0.8
    z[torch.from_numpy(~valid)] = float("nan")
    z[3], valid[3] = -torch.inf, True                       # nothing
    z[4], valid[4] = -torch.inf, True
    z[4, 17] = -3                                           # one expert
    z[5, :24], valid[5] = -torch.inf, True                  # three groups of six
    z[6], valid[6] = torch.finfo(DT[dtype]).min, True       # a type's lowest value is a score
    z[7], valid[7] = -200.0, True                           # scores that fp32 cannot hold
    z[8], valid[8] = -200.0, True
    z[8, ::5] = 90.0
    bias = g.standard_normal(E) * 0.1
    bias[[2, 9, 30]] = np.nan, np.inf, -np.inf
    b = bias if biased else None
    for normalize in (True, False):
        for groups, top, best in ((1, 1, 2), (8, 3, 2), (8, 2, 1)):
            check(z.to(DEV), k, kind, b, groups, top, best, normalize, 1.7, valid, 8)
    z[10, 7], z[11, 8] = float("nan"), float("inf")
    valid[10:12] = True
    r, _ = check(z.to(DEV), k, kind, b, 8, 3, 2, True, 1.7, valid, 8)
    assert (r.idx[10:12] == -1).all() and r.weight[10:12].isnan().all()


def test_no_tokens():
    r = mxq.mx_route_scored(torch.empty((0, 64), device=DEV), 4, bias=torch.zeros(64, device=DEV), groups=8, top_groups=2)
    assert not r.counts.any() and not r.offs.any() and int(r.live) == 0 and float(r.loss) == 0 and not r.prob.any()


# Equal logits with equal biases are equal: the lowest experts and groups.
@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k,groups,top", [(16, 5, 4, 2), (64, 8, 8, 3), (256, 8, 8, 4), (1024, 16, 32, 9), (100, 7, 5, 3)])
def test_ties(E, k, groups, top, kind):
    g = np.random.default_rng(E)
    z = torch.from_numpy(g.integers(-3, 4, (150, E)) * 0.5).float().to(DEV)
    z[0] = 0.25
    for bias in (None, np.zeros(E), np.full(E, 0.3), np.repeat(g.integers(0, 3, groups) * 0.125, E // groups)):
        check(z, k, kind, bias, groups, top, 2)
        check(z, k, kind, bias, groups, top, 1)
        check(z, k, kind, bias)


# Scores and biases whose sums differ far below fp32's digits, in either
# direction, between picks, at the last pick and its successor, and everywhere.
@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k", [(16, 4), (60, 8), (256, 8), (256, 16), (600, 8), (1024, 16)])
def test_sums_that_differ_below_fp32(E, k, kind):
    g = np.random.default_rng(E + k)
    T = 90
    z = np.float32(g.standard_normal((1, E)))
    s = so.scores(z[0].astype(np.float64), kind)
    # biases that bring every score to a level up to its own rounding: u differ by 2^-25 or so
    level = np.where(g.random(E) < 0.5, 0.75, 0.75 - 0.01 * g.random(E))
    bias = np.float32(level - s).astype(np.float64)
    u = s + bias
    gaps = np.diff(np.sort(u))
    assert gaps[gaps > 0].min() < 1e-7 and gaps.min() > 4e-15         # closer than fp32 tells, wider than binary64 errs
    zz = torch.from_numpy(np.repeat(z, T, 0)).to(DEV)
    zz[1::3] = torch.from_numpy(np.float32(g.standard_normal((T // 3, E)))).to(DEV)
    check(zz, k, kind, bias)
    if E % 4 == 0:
        check(zz, k, kind, bias, 4, 2, 2)


# Worths of groups that differ below fp32's digits.
@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("biased", [False, True])
def test_groups_that_differ_below_fp32(kind, biased):
    g = np.random.default_rng(11)
    T, groups, size = 80, 16, 8
    z = g.standard_normal((T, groups, size)) * 0.3 - 3
    z[:, :, 0], z[:, :, 1] = 1.5, 1.25                                # the two best of every group alike
    z = np.float32(z)
    z[:, ::3, 1] = np.nextafter(z[:, ::3, 1], np.float32(9))          # an ulp more in some
    z[:, 1::5, 0] = np.nextafter(z[:, 1::5, 0], np.float32(-9))
    z = g.permuted(z, axis=2).reshape(T, groups * size)
    bias = np.zeros(groups * size) + 0.1 if biased else None
    for top in (1, 5, 15):
        check(torch.from_numpy(z).to(DEV), 8, kind, bias, groups, top, 2)
        check(torch.from_numpy(z).to(DEV), 8, kind, bias, groups, top, 1)


# Biases far larger than scores, of either sign, and equal but for a few.
@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("size", [1e-6, 3.0, 1e4, 1e12, 1e37])
def test_biases_of_any_size(size, kind):
    g = np.random.default_rng(13)
    z = logits(100, 64, "f32", g)
    check(z, 8, kind, g.standard_normal(64) * size, 8, 3, 2)
    check(z, 8, kind, np.where(g.random(64) < 0.8, 1.0, g.standard_normal(64)) * size, 8, 8, 2)


def test_peaked_and_saturated_scores():
    """Softmax rows whose picks' probabilities are far below fp32's digits of the
    largest; sigmoid rows past the logit where fp32 scores are all 1."""
    g = np.random.default_rng(17)
    z = np.float32(g.standard_normal((120, 128)))
    z[np.arange(120), g.integers(0, 128, 120)] += 40
    for bias in (None, g.standard_normal(128) * 1e-9):
        check(torch.from_numpy(z).to(DEV), 8, "softmax", bias, 8, 3, 2)
    z = np.float32(g.standard_normal((120, 128)) * 0.5 + 20)
    for bias in (None, g.standard_normal(128) * 1e-9, np.zeros(128)):
        check(torch.from_numpy(z).to(DEV), 8, "sigmoid", bias, 8, 3, 2)


# ------------------------------------------------------------------ gradient
@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (37, 16, 16), (130, 60, 6), (300, 256, 8), (70, 500, 8), (40, 1024, 16), (9, 5, 1)])
def test_gradient(T, E, k, normalize, dtype, kind):
    g = np.random.default_rng(T + E + k)
    z = logits(T, E, dtype, g)
    valid = g.random(T) < 0.9
    valid[0] = True
    z[torch.from_numpy(~valid).to(DEV)] = float("nan")
    if T > 20:
        z[3], valid[3] = -torch.inf, True
        z[5, 1], valid[5] = float("nan"), True
    bias = g.standard_normal(E) * 0.05
    dw, dl = g.standard_normal((T, k)), np.array([0.37])
    v = dev(valid, torch.bool)
    r = mxq.mx_route_scored(z, k, bias=dev(bias), score=kind, normalize=normalize, scale=2.5, valid=v, align=1)
    b = bias.astype(np.float32).astype(np.float64)
    want = so.route(f64(z), k, kind, b, normalize=normalize, scale=2.5, valid=valid, M=r.rows)
    dwd, dld = dev(dw), dev(dl)
    z64, dw64, dl64 = f64(z), f64(dwd), float(dld)
    buf = torch.full((T, E + 3), 99.0, dtype=DT[dtype], device=DEV)
    for w_, l_ in ((dwd, dld), (dwd, None), (None, dld), (None, None)):
        got = mxq.mx_route_scored_grad(z, r, w_, l_, v, out=buf[:, :E])
        ref, mag = so.grad(z64, want, k, kind, normalize, 2.5, dw64 if w_ is not None else dw64 * 0,
                           dl64 if l_ is not None else 0.0)
        err = mag * (12 * want["spread"] + 6 * E + 6 * k + 96) * U + 2.0 ** -100
        if dtype == "bf16":
            err = err + 2.0 ** -8 * (np.abs(ref) + err)
        bad = ~(np.abs(f64(got) - ref) <= err) & ~(np.isnan(f64(got)) & np.isnan(ref))
        assert not bad.any(), (np.argwhere(bad)[0], f64(got)[bad][0], ref[bad][0], err[bad][0])
        assert (buf[:, E:] == 99).all()


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
def test_the_only_pick_of_a_normalized_routing_has_no_gradient(kind):
    """But for the 1e-20: s / (s + 1e-20) has the slope 1e-20 / (s + 1e-20)^2, and
    the best of 24 softmax scores is 1 / 24 at least, of sigmoid ones 0.5 here;
    times s (1 - s) or s, which is less than s: 24e-20 of dweight at most."""
    z = torch.randn((50, 24), device=DEV)
    z[:, 3] = z[:, 3].abs()
    dw = torch.randn((50, 1), device=DEV)
    r = mxq.mx_route_scored(z, 1, score=kind)
    d = mxq.mx_route_scored_grad(z, r, dw)
    assert (d.double().abs() <= 24.1e-20 * dw.double().abs()).all()


def test_gradient_of_many_tokens():
    """More tokens than the gradient's grid takes at once."""
    T, E, k = 70001, 12, 3
    z = torch.randn((T, E), device=DEV) * 2
    r = mxq.mx_route_scored(z, k, normalize=True, scale=1.0)
    dw = torch.randn((T, k), device=DEV)
    got = mxq.mx_route_scored_grad(z, r, dw).double()
    zz = z.double().requires_grad_()
    s = torch.sigmoid(zz).gather(1, r.idx.long())
    (s / s.sum(1, keepdim=True) * dw.double()).sum().backward()
    assert (got - zz.grad).abs().max() < (12 * 16 + 6 * E + 6 * k + 96) * U * 4 * float(dw.abs().max())


# ---------------------------------------------------------------- bias's step
@pytest.mark.parametrize("E", [1, 5, 64, 1000, 1024])
def test_bias_step(E):
    g = np.random.default_rng(E)
    bias = torch.from_numpy(g.standard_normal(E)).float().to(DEV)
    for counts in (g.integers(0, 5, E), np.full(E, 7), g.integers(0, 2 ** 31 - 1, E)):
        c = torch.from_numpy(counts.astype(np.int32)).to(DEV)
        sign = torch.from_numpy(np.sign(int(counts.sum()) - counts.astype(object) * E).astype(np.float32)).to(DEV)
        want = bias + 0.125 * sign
        assert torch.equal(mxq.mx_route_bias_step(bias, c, 0.125), want)
        b = bias.clone()
        assert mxq.mx_route_bias_step(b, c, 0.125, out=b) is b and torch.equal(b, want)


def test_the_bias_evens_the_counts():
    """Steps of the bias against experts that are liked unequally."""
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    liked = torch.randn(32, generator=g, device=DEV)
    bias, spread = torch.zeros(32, device=DEV), []
    for _ in range(300):
        z = torch.randn((1024, 32), generator=g, device=DEV) + liked
        r = mxq.mx_route_scored(z, 4, bias=bias, groups=4, top_groups=2)
        spread.append(float(r.counts.float().std()))
        mxq.mx_route_bias_step(bias, r.counts, 0.004, out=bias)
    assert sum(spread[-20:]) < 0.25 * sum(spread[:20])


def test_logits_far_apart():
    """Rows 2^23 elements apart: offsets past 32 bits, the bits of contiguous rows."""
    g = torch.Generator(device=DEV)
    g.manual_seed(23)
    T, E, k = 300, 64, 4
    z = torch.randn((T, E), generator=g, device=DEV).bfloat16()
    far, out = (torch.empty((T, 1 << 23), dtype=torch.bfloat16, device=DEV)[:, 5:E + 5] for _ in range(2))
    far.copy_(z)
    bias = 0.1 * torch.randn(E, generator=g, device=DEV)
    dw = torch.randn((T, k), generator=g, device=DEV)
    a, b = (mxq.mx_route_scored(x, k, bias, groups=4, top_groups=2) for x in (z, far))
    for name in ("idx", "weight", "slot", "src", "counts", "offs", "live", "prob", "loss"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name
    want = mxq.mx_route_scored_grad(z, a, dw, torch.ones(1, device=DEV))
    mxq.mx_route_scored_grad(far, b, dw, torch.ones(1, device=DEV), out=out)
    assert torch.equal(out, want)


# ------------------------------------------------------- state, graphs, refusals
def test_routings_are_told_apart():
    z = torch.randn((40, 16), device=DEV)
    plan = mxq.mx_routing(40, 16, 4, align=1, device=DEV)
    dw = torch.randn((40, 4), device=DEV)
    r = mxq.mx_route_scored(z, out=plan, scale=2.0)
    assert r.generation == 1 and r.scored == ("sigmoid", 2.0) and r.normalize and not r.masked
    with pytest.raises(ValueError):
        mxq.mx_route_grad(z, r, dw)
    mxq.mx_route(z, out=plan)
    assert plan.scored is None and plan.generation == 2
    with pytest.raises(ValueError):
        mxq.mx_route_scored_grad(z, plan, dw)
    mxq.mx_route_scored(z, valid=torch.ones(40, dtype=torch.bool, device=DEV), out=plan)
    with pytest.raises(ValueError):
        mxq.mx_route_scored_grad(z, plan, dw)                        # without the mask
    with pytest.raises(ValueError):
        mxq.mx_route_scored_grad(z, plan, dw, valid=torch.ones(40, dtype=torch.bool, device=DEV), generation=2)
    with pytest.raises(AttributeError):
        plan.scored = None


def test_refusals_of_the_binding():
    z, b = torch.randn((8, 24), device=DEV), torch.zeros(24, device=DEV)
    plan = mxq.mx_routing(8, 24, 7, align=1, device=DEV)
    for kw in (dict(score="tanh"), dict(groups=5), dict(groups=0), dict(groups=4, top_groups=5), dict(groups=4, top_groups=0),
               dict(group_best=3), dict(bias=b[:23]), dict(bias=b.double()), dict(bias=b.cpu()), dict(groups=4, top_groups=1, k=7),
               dict(groups=4, top_groups=1, out=plan), dict(k=0), dict(k=17), dict(valid=torch.ones(7, device=DEV) > 0)):
        kw = {"k": None if "out" in kw else 2, **kw}
        with pytest.raises(ValueError):
            mxq.mx_route_scored(z, **kw)
    with pytest.raises(ValueError):
        mxq.mx_route_scored(z)                                       # neither k nor out
    for args in ((b, torch.zeros(23, dtype=torch.int32, device=DEV)), (b, torch.zeros(24, device=DEV)),
                 (b.double(), torch.zeros(24, dtype=torch.int32, device=DEV)), (b.cpu(), torch.zeros(24, dtype=torch.int32))):
        with pytest.raises(ValueError):
            mxq.mx_route_bias_step(*args, 0.1)


def test_a_step_in_a_graph():
    """Routing, its gradient and the bias's step in place, captured and replayed
    with new logits, while an eager routing is alive."""
    T, E, k = 300, 64, 6
    z, dw = torch.randn((T, E), device=DEV), torch.randn((T, k), device=DEV)
    plan, twin = (mxq.mx_routing(T, E, k, align=16, device=DEV) for _ in range(2))
    kw = dict(score="sigmoid", groups=8, top_groups=3)

    def step(plan, bias):
        r = mxq.mx_route_scored(z, bias=bias, out=plan, **kw)
        d = mxq.mx_route_scored_grad(z, r, dw)
        mxq.mx_route_bias_step(bias, r.counts, 0.01, out=bias)
        return d

    bias, other = torch.zeros(E, device=DEV), torch.zeros(E, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(plan, bias)
    torch.cuda.current_stream().wait_stream(side)
    bias.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(plan, bias)
    for rep in range(4):
        z.copy_(torch.randn((T, E), device=DEV))
        held.fill_(rep)
        graph.replay()
        want = step(twin, other)
        torch.cuda.synchronize()
        assert torch.equal(held, want) and torch.equal(bias, other) and bias.any()
        for n in ("idx", "weight", "slot", "src", "counts", "offs", "live", "prob", "loss"):
            assert torch.equal(getattr(plan, n), getattr(twin, n)), n


def test_the_same_inputs_give_the_same_bits_on_two_streams():
    z = [torch.randn((5000, 128), device=DEV) for _ in range(2)]
    bias = torch.randn(128, device=DEV) * 0.05
    call = lambda i: mxq.mx_route_scored(z[i], 8, bias=bias, groups=8, top_groups=4)  # noqa: E731
    want = [call(0), call(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in z]
    got = []
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append(call(i))
    torch.cuda.synchronize()
    for i, r in enumerate(got):
        for n in ("idx", "weight", "slot", "src", "counts", "prob", "loss"):
            assert torch.equal(getattr(r, n), getattr(want[i % 2], n)), n
