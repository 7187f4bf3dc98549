"""CPU-only checks of the scored-routing part of the C ABI: declared functions
are exported, arguments are refused on the host, and the binary64 gradient
agrees with differences of its own forward."""
import os
import re

import numpy as np
import pytest

import mx9_dual_axis_amd as mxq
import scored_oracle as so
from mx9_dual_axis_amd import routed

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20           # never dereferenced: every call below is refused or empty
NULL, DTYPE, MODE, SHAPE, STRIDE, ALIGN, OVERLAP = 1, 2, 4, 5, 6, 7, 8


def at(i):
    return FAKE * (16 + 16 * i)


def lib():
    return routed._L()


def test_every_declared_function_is_exported():
    src = open(os.path.join(ROOT, "include", "mxq_scored.h")).read()
    names = re.findall(r"^\s*(?:int|int64_t)\s+(\w+)\s*\(", re.sub(r"/\*.*?\*/", "", src, flags=re.S), flags=re.M)
    assert len(names) == 3
    for n in names:
        assert hasattr(lib(), n) and callable(getattr(mxq, n)), n
    assert {k.lower(): int(v) for k, v in re.findall(r"MX_SCORE_(\w+) = (\d)", src)} == routed.SCORES


def route(**kw):
    a = dict(z=at(0), dt=0, T=70, E=24, ld=24, valid=at(1), bias=at(2), score=0, groups=4, top=2, best=2, k=3, norm=1, scale=1.0,
             align=1, M=210, idx=at(3), w=at(4), slot=at(5), src=at(6), counts=at(7), offs=at(8), live=at(9), prob=at(10),
             loss=at(11), ws=at(12), size=1 << 20)
    a.update(kw)
    return lib().mx_route_scored(*a.values(), None)


def test_route_refusals():
    for n in ("z", "idx", "w", "slot", "src", "counts", "offs", "live", "prob", "loss", "ws"):
        assert route(**{n: None}) == NULL, n
    assert route(dt=2) == DTYPE and route(score=2) == MODE and route(score=-1) == MODE
    for kw in (dict(T=-1), dict(E=0), dict(E=1025, ld=1025), dict(k=0), dict(k=17), dict(align=0), dict(M=209), dict(size=8),
               dict(groups=0), dict(groups=5), dict(groups=33, E=66, ld=66), dict(top=0), dict(top=5), dict(best=0), dict(best=3),
               dict(top=1, k=7, M=490)):
        assert route(**kw) == SHAPE, kw
    assert route(ld=23) == STRIDE
    for n in ("z", "bias", "idx", "w", "slot", "src", "counts", "offs", "live", "prob", "loss", "ws"):
        assert route(**{n: at(20) + 2}) == ALIGN, n
    for n in ("idx", "w", "slot", "src", "counts", "offs", "live", "prob", "loss", "ws"):
        for m in ("z", "valid", "bias"):
            assert route(**{n: at(20), m: at(20)}) == OVERLAP, (n, m)
    assert route(w=at(3) + 4) == OVERLAP and route(loss=at(9)) == OVERLAP


def grad(**kw):
    a = dict(z=at(0), dt=0, T=70, E=24, ld=24, valid=at(1), score=1, k=3, norm=1, scale=1.0, idx=at(3), dw=at(4), counts=at(5),
             live=at(6), dl=at(7), d=at(8), ldd=24)
    a.update(kw)
    return lib().mx_route_scored_grad(*a.values(), None)


def test_gradient_refusals():
    for n in ("z", "idx", "counts", "live", "d"):
        assert grad(**{n: None}) == NULL, n
    assert grad(dt=3) == DTYPE and grad(score=2) == MODE and grad(T=-1) == SHAPE and grad(k=0) == SHAPE and grad(k=25) == SHAPE
    assert grad(ld=23) == STRIDE and grad(ldd=23) == STRIDE
    for n in ("z", "idx", "dw", "counts", "live", "dl", "d"):
        assert grad(**{n: at(20) + 2}) == ALIGN, n
    for n in ("z", "valid", "idx", "dw", "counts", "live", "dl"):
        assert grad(d=at(20), **{n: at(20)}) == OVERLAP, n
    assert grad(T=0, z=None, idx=None, counts=None, live=None, d=None) == 0


def test_bias_step_refusals():
    f = lib().mx_route_bias_step
    assert f(None, at(1), 8, 0.1, at(2), None) == NULL and f(at(0), None, 8, 0.1, at(2), None) == NULL
    assert f(at(0), at(1), 8, 0.1, None, None) == NULL
    assert f(at(0), at(1), 0, 0.1, at(2), None) == SHAPE and f(at(0), at(1), 1025, 0.1, at(2), None) == SHAPE
    assert f(at(0) + 2, at(1), 8, 0.1, at(2), None) == ALIGN
    assert f(at(0), at(1), 8, 0.1, at(1), None) == OVERLAP and f(at(0), at(1), 8, 0.1, at(0) + 4, None) == OVERLAP


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("normalize", [True, False])
def test_gradient_against_differences(kind, normalize):
    """The binary64 gradient that the GPU tests compare with."""
    g = np.random.default_rng(2)
    T, E, k, scale = 5, 12, 3, 2.5
    z = g.standard_normal((T, E)) * 1.5
    z[1, 4] = -np.inf
    valid = np.array([True, True, False, True, True])
    bias = g.standard_normal(E) * 0.05
    kw = dict(bias=bias, groups=3, top=2, best=2, normalize=normalize, scale=scale, valid=valid, M=T * k)
    r = so.route(z, k, kind, **kw)
    dw, dl = g.standard_normal((T, k)), 0.7

    def f(z):
        q = so.route(z, k, kind, **kw)
        assert np.array_equal(q["idx"], r["idx"])
        return (q["weight"] * dw).sum() + dl * q["loss"]

    d, mag = so.grad(np.where(valid[:, None], z, -np.inf), r, k, kind, normalize, scale, dw, dl)
    h = 1e-6
    for t in range(T):
        for e in range(E):
            if z[t, e] == -np.inf:
                assert d[t, e] == 0
                continue
            zp, zm = z.copy(), z.copy()
            zp[t, e] += h
            zm[t, e] -= h
            assert abs((f(zp) - f(zm)) / (2 * h) - d[t, e]) < 1e-7
            assert abs(d[t, e]) <= mag[t, e] * (1 + 1e-12)
