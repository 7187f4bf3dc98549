"""GPU tests of scored routing where scores are close to each other, or too
small for fp32: picks as binary64 decides them (scored_oracle, through the
comparison that test_gpu_scored makes)."""
import numpy as np
import pytest
import torch

import mx9_dual_axis_amd as mxq
import scored_oracle as so
from helpers import require_gpu, say
from test_gpu_scored import DEV, DT, check

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(request):
    require_gpu()
    say(request.node.name)


# What picks go by spans next to nothing: a step of the keys' grid is below
# fp32's least normal number, or its inverse above the largest.
@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("span", [1e-29, 1e-31, 2e-32, 1e-32, 1e-33, 1e-38, 1e-42])
def test_logits_that_span_next_to_nothing(span, kind):
    g = np.random.default_rng(29)
    for row, k in (([0, 0, 1, 0], 3), ([0, 0, 1, 0], 1), ([0, 1], 2), ([1, 0], 2), ([0.25, 1, 0.5, 0.75], 2)):
        z = torch.tensor(row, dtype=torch.float64).mul(span).float().repeat(5, 1).to(DEV)
        check(z, k, kind)
    for E, k in ((16, 4), (60, 8), (256, 8), (600, 16)):
        for dtype in ("f32", "bf16"):
            z = torch.from_numpy(g.random((70, E)) * span).to(DT[dtype])
            z[3:, 1:E:7] = 0.0
            z[5:, 2:E:5] = -torch.inf
            z[7:40, E // 4:] = -torch.inf                                 # few experts
            check(z.to(DEV), k, kind)
            if E % 4 == 0:
                check(z.to(DEV), k, kind, None, 4, 2, 2)


@pytest.mark.parametrize("level", [-60.0, -73.0, -80.0, -83.0, -95.0])
@pytest.mark.parametrize("E,k", [(2, 2), (4, 3), (16, 4), (256, 8)])
def test_sigmoid_scores_next_to_nothing_with_a_bias(E, k, level):
    """Biases of 0: u is the score itself.  (Below 2^-126 scores may be 0, which
    shows in prob, whose sum has no more than 1e-20 added: picks alone there.)"""
    g = np.random.default_rng(E)
    z = np.float32(level + 0.5 * g.standard_normal((70, E)))
    for bias in (np.zeros(E), np.where(np.arange(E) % 5 == 4, -np.inf, 0.0)):
        for groups, top in ((1, 1), (4, 2)) if E >= 16 else ((1, 1),):
            if level > -90:
                check(torch.from_numpy(z).to(DEV), k, "sigmoid", bias, groups, top)
                continue
            r = mxq.mx_route_scored(torch.from_numpy(z).to(DEV), k, torch.from_numpy(bias).float().to(DEV), groups=groups,
                                    top_groups=top, align=1)
            want = so.route(z.astype(np.float64), k, "sigmoid", bias, groups, top, align=1, M=r.rows)
            assert np.array_equal(r.idx.cpu().numpy(), want["idx"])


@pytest.mark.parametrize("top", [60.0, 75.0, 86.0, 100.0])
@pytest.mark.parametrize("E,k", [(3, 2), (16, 4), (256, 8)])
def test_softmax_scores_next_to_nothing_with_a_bias(E, k, top):
    """The largest score's expert is barred by its bias; the others' are e^-top of it."""
    g = np.random.default_rng(E)
    z = np.float32(g.standard_normal((70, E)))
    z[:, 0] = top
    check(torch.from_numpy(z).to(DEV), k, "softmax", np.where(np.arange(E) == 0, -np.inf, 0.0))


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("best", [1, 2])
def test_worths_of_scores_that_fp32_loses(best, kind):
    """Groups whose scores are about fp32's least normal number, some above and
    some below it, without a bias: worths are sums of what binary64 has."""
    g = np.random.default_rng(31)
    high = 1.0 if kind == "sigmoid" else 0.0                          # (scores of 0.73, of a quarter)
    z = np.full((300, 16), -120.0)
    z[:, :4] = high
    z[0, 4], z[0, 5], z[0, 8] = -87.0, -87.4, -86.9
    z[1, 8], z[1, 9], z[1, 4] = -87.0, -87.4, -86.9
    low = g.uniform(-89.5, -85.5, (298, 12))
    z[2:, 4:] = np.where(g.random((298, 12)) < 0.6, low, z[2:, 4:])
    z = np.float32(z)
    for k, top in ((6, 2), (8, 3), (4, 2)):
        check(torch.from_numpy(z).to(DEV), k, kind, None, 4, top, best)
        check(torch.from_numpy(z).to(DEV), k, kind, None, 8, top + 1, best)


def test_picks_of_a_group_that_is_found_again():
    """Two groups whose worths only binary64 tells apart, the other one first; in
    it two experts whose biases of some -1000 bring their sums within 2e-8 of the
    same halfway point between fp32 numbers, which lie 6e-5 apart there."""
    g = np.random.default_rng(37)
    T, step = 3000, 2.0 ** -14
    bias = np.array([0.0, -1, -1, -1, 0, -1000, -1000 - 6554 * step, -3000])
    mid = (np.floor(g.uniform(0.15, 0.45, T) / step) + 0.5) * step
    logit = lambda s: np.log(s / (1 - s))  # noqa: E731
    z = g.standard_normal((T, 8))
    z[:, 0], z[:, 4] = 0.0, 4e-9                                      # scores of 0.5 and 1e-9 more
    z[:, 5], z[:, 6] = logit(mid), logit(mid + 6554 * step)
    check(torch.from_numpy(z).float().to(DEV), 2, "sigmoid", bias, 2, 1, 1)
    check(torch.from_numpy(z).float().to(DEV), 3, "sigmoid", bias, 2, 1, 1)


def test_shares_of_scores_far_from_zero():
    """One token, one large score: the others' shares are their own scores.  A
    score is within 16 u of itself whatever its logit (scored_oracle; the wider
    bound of test_gpu_scored's comparison is of scores whose argument was rounded), so is the
    sum; two additions of what is no more than 2^-60 of it, a reciprocal and a
    product: 36 u."""
    g = np.random.default_rng(41)
    for E in (64, 256, 1000):
        z = np.float32(g.uniform(-85, -60, (1, E)))
        z[0, 3] = 20.0
        s = so.scores(z[0].astype(np.float64), "sigmoid")
        share = s / (s.sum() + so.EPS)
        got = mxq.mx_route_scored(torch.from_numpy(z).to(DEV), 4, align=1).prob.double().cpu().numpy()
        assert (np.abs(got - share) <= 36 * so.U * share).all(), (np.abs(got - share) / share / so.U).max()
