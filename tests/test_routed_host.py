"""CPU-only checks of the routed-expert part of the C ABI: declared functions
are exported, arguments are refused on the host, and the plain numpy forms that
the GPU tests compare with agree with differences of their own forward."""
import os
import re

import numpy as np
import pytest
import torch

import mx9_dual_axis_amd as mxq
import routed_oracle as ro
from mx9_dual_axis_amd import routed

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20           # never dereferenced: every call below is refused or empty
NULL, DTYPE, SHAPE, STRIDE, ALIGN, OVERLAP = 1, 2, 5, 6, 7, 8


def at(i):
    return FAKE * (16 + 16 * i)


def lib():
    return routed._L()


def test_every_declared_function_is_exported():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "mxq_routed.h")).read(), flags=re.S)
    names = re.findall(r"^\s*(?:int|int64_t)\s+(\w+)\s*\(", src, flags=re.M)
    assert len(names) == 13
    for n in names:
        assert hasattr(lib(), n), n


@pytest.mark.parametrize("T,E,k,align", [(0, 1, 1, 1), (1, 64, 4, 1), (37, 10, 3, 128), (1000, 16, 16, 128), (3, 1024, 2, 7)])
def test_row_bound(T, E, k, align):
    M = lib().mx_route_rows(T, E, k, align)
    assert M == ro.rows_needed(T, E, k, align)
    # the worst case: every expert of the first picks gets one pick more than whole groups
    picks, groups = T * k, min(E, T * k)
    worst = 0
    if groups:
        sizes = [1] * groups
        sizes[0] += picks - groups
        worst = sum(-(-s // align) * align for s in sizes)
    assert worst <= M


def test_row_bound_refusals():
    for a in [(-1, 8, 2, 1), (4, 0, 1, 1), (4, 1025, 1, 1), (4, 8, 0, 1), (4, 8, 9, 1), (4, 64, 17, 1), (4, 8, 2, 0),
              (4, 8, 2, 65537), (1 << 30, 8, 2, 1)]:
        assert lib().mx_route_rows(*a) == -1, a
    assert lib().mx_route_workspace(64, 256) == 0
    assert lib().mx_route_workspace(65, 256) > 0
    assert lib().mx_route_workspace(-1, 8) == -1
    assert lib().i8_linear_workspace(3, 17) >= 3 * 32 + 12
    assert lib().i8_linear_workspace(1, 131072) == -1


def _route(**kw):
    a = dict(logits=at(0), dtype=1, T=100, E=8, ld=8, valid=None, k=2, norm=1, align=16, M=320, idx=at(1), weight=at(2),
             slot=at(3), src=at(4), counts=at(5), offs=at(6), live=at(7), prob=at(8), loss=at(9), ws=at(10), wsb=1 << 16)
    a.update(kw)
    return lib().mx_route(*a.values(), None)


def test_route_refusals():
    for n in ("logits", "idx", "weight", "slot", "src", "counts", "offs", "live", "prob", "loss", "ws"):
        assert _route(**{n: None}) == NULL, n
    assert _route(dtype=2) == DTYPE
    for kw in (dict(T=-1), dict(E=0), dict(E=2000, ld=2000), dict(k=0), dict(k=9), dict(align=0), dict(M=319),
               dict(M=(1 << 30) + 16), dict(wsb=100)):
        assert _route(**kw) == SHAPE, kw
    assert _route(ld=7) == STRIDE
    assert _route(logits=at(0) + 1) == ALIGN and _route(slot=at(3) + 2) == ALIGN and _route(ws=at(10) + 2) == ALIGN
    assert _route(slot=at(1) + 4) == OVERLAP             # two outputs
    assert _route(src=at(0) + 8) == OVERLAP              # an output in an input
    assert _route(valid=at(9)) == OVERLAP
    assert _route(ws=at(4) + 64) == OVERLAP


def _route_grad(**kw):
    a = dict(logits=at(0), dtype=0, T=100, E=8, ld=8, valid=None, k=2, norm=1, idx=at(1), weight=at(2), dw=at(3),
             counts=at(4), live=at(5), dloss=at(6), out=at(7), ld_d=8)
    a.update(kw)
    return lib().mx_route_grad(*a.values(), None)


def test_route_grad_refusals():
    for n in ("logits", "idx", "weight", "counts", "live", "out"):
        assert _route_grad(**{n: None}) == NULL, n
    assert _route_grad(dtype=7) == DTYPE
    assert _route_grad(k=9) == SHAPE and _route_grad(E=0) == SHAPE
    assert _route_grad(ld=7) == STRIDE and _route_grad(ld_d=7) == STRIDE
    assert _route_grad(out=at(7) + 2) == ALIGN and _route_grad(dw=at(3) + 1) == ALIGN
    assert _route_grad(out=at(0)) == OVERLAP and _route_grad(out=at(3) + 16) == OVERLAP
    assert _route_grad(T=0, logits=None, out=None) == 0


def test_dispatch_refusals():
    def d(**kw):
        a = dict(x=at(0), dtype=1, T=10, N=64, ld=64, slot=at(1), src=at(2), k=2, M=20, out=at(3), ld_o=64)
        a.update(kw)
        return lib().mx_dispatch(*a.values(), None)

    for n in ("x", "slot", "src", "out"):
        assert d(**{n: None}) == NULL, n
    assert d(dtype=3) == DTYPE
    for kw in (dict(T=-1), dict(N=-1), dict(M=-1), dict(k=0), dict(k=65), dict(M=1 << 31), dict(T=1 << 30)):
        assert d(**kw) == SHAPE, kw
    assert d(ld=63) == STRIDE and d(ld_o=63) == STRIDE and d(ld_o=1 << 50) == STRIDE
    assert d(x=at(0) + 1) == ALIGN and d(src=at(2) + 2) == ALIGN
    assert d(out=at(0) + 64) == OVERLAP and d(out=at(1)) == OVERLAP
    assert d(N=0, x=None, out=None) == 0 and d(M=0, src=None, out=None) == 0


def test_quantize_refusals():
    def d(**kw):
        a = dict(x=at(0), dtype=1, T=10, K=64, ld=64, slot=at(1), src=at(2), k=2, M=20, q=at(3), ld_q=64, s=at(4))
        a.update(kw)
        return lib().mx_dispatch_i8(*a.values(), None)

    def r(**kw):
        a = dict(x=at(0), dtype=0, T=10, K=64, ld=64, q=at(3), ld_q=64, s=at(4))
        a.update(kw)
        return lib().i8_quantize_rows(*a.values(), None)

    for n in ("x", "slot", "src", "q", "s"):
        assert d(**{n: None}) == NULL, n
    for n in ("x", "q", "s"):
        assert r(**{n: None}) == NULL, n
    assert d(dtype=2) == DTYPE and r(dtype=2) == DTYPE
    assert d(k=0) == SHAPE and r(T=-1) == SHAPE and r(T=1 << 26) == SHAPE
    assert d(ld=1) == STRIDE and d(ld_q=63) == STRIDE and r(ld_q=63) == STRIDE
    assert d(s=at(4) + 1) == ALIGN and r(x=at(0) + 2) == ALIGN
    assert d(s=at(3) + 8) == OVERLAP and r(q=at(0) + 16) == OVERLAP
    assert r(T=0, x=None, q=None, s=None) == 0


def _gemm(**kw):
    a = dict(A=at(0), lda=64, sA=at(1), B=at(2), ldb=64, sB=at(3), bias=None, M=10, N=20, K=64, C=at(5), ldc=20, dt=1)
    a.update(kw)
    return lib().i8_gemm_nt(*a.values(), None)


def test_gemm_refusals():
    for n in ("A", "sA", "B", "sB", "C"):
        assert _gemm(**{n: None}) == NULL, n
    assert _gemm(dt=2) == DTYPE
    for kw in (dict(M=-1), dict(N=-1), dict(K=-1), dict(K=131072, lda=1 << 18, ldb=1 << 18), dict(M=(1 << 30) + 1),
               dict(M=1 << 30, N=1 << 30, ldc=1 << 30)):
        assert _gemm(**kw) == SHAPE, kw
    assert _gemm(lda=63) == STRIDE and _gemm(ldb=63) == STRIDE and _gemm(ldc=19) == STRIDE
    assert _gemm(lda=1 << 50) == STRIDE
    assert _gemm(sA=at(1) + 2) == ALIGN and _gemm(bias=at(4) + 1) == ALIGN and _gemm(C=at(5) + 1) == ALIGN
    for n, p in (("A", at(5) + 10), ("sA", at(5)), ("B", at(5) + 32), ("sB", at(5) + 4), ("bias", at(5) + 8)):
        assert _gemm(**{n: p}) == OVERLAP, n
    assert _gemm(M=0, A=None, C=None) == 0 and _gemm(N=0, B=None, C=None) == 0


def test_linear_refusals():
    def r(**kw):
        a = dict(x=at(0), dtype=1, ld=64, B=at(2), ldb=64, sB=at(3), bias=None, M=10, N=20, K=64, C=at(5), ldc=20, dt=0,
                 ws=at(6), wsb=1 << 12)
        a.update(kw)
        return lib().i8_linear(*a.values(), None)

    for n in ("x", "B", "sB", "C", "ws"):
        assert r(**{n: None}) == NULL, n
    assert r(dtype=2) == DTYPE and r(dt=2) == DTYPE
    assert r(wsb=100) == SHAPE and r(K=131072) == SHAPE
    assert r(ld=63) == STRIDE and r(ldb=1) == STRIDE
    assert r(ws=at(6) + 8) == ALIGN and r(x=at(0) + 1) == ALIGN
    assert r(ws=at(0) + 16) == OVERLAP and r(C=at(6) + 16) == OVERLAP and r(ws=at(2)) == OVERLAP
    assert r(bias=at(5)) == OVERLAP and r(bias=at(6)) == OVERLAP
    assert r(M=0, x=None, ws=None, C=None) == 0


def test_grouped_refusals():
    def r(**kw):
        a = dict(A=at(0), lda=64, sA=at(1), B=at(2), ldb=64, b_gs=20 * 64, sB=at(3), sb_gs=20, offs=at(4), G=4, M=10,
                 N=20, K=64, C=at(5), ldc=20, dt=1)
        a.update(kw)
        return lib().i8_grouped_gemm_rows(*a.values(), None)

    for n in ("A", "sA", "B", "sB", "offs", "C"):
        assert r(**{n: None}) == NULL, n
    assert r(G=0) == SHAPE and r(K=131072) == SHAPE
    assert r(b_gs=-1) == STRIDE and r(sb_gs=-1) == STRIDE and r(b_gs=1 << 50) == STRIDE
    assert r(offs=at(4) + 2) == ALIGN
    assert r(C=at(2) + 3 * 20 * 64) == OVERLAP           # inside the last group's operand
    assert r(C=at(4)) == OVERLAP
    assert r(M=0) == 0


def test_combine_refusals():
    def c(**kw):
        a = dict(rows=at(0), dtype=1, M=20, N=64, ld=64, slot=at(1), weight=at(2), k=2, T=10, y=at(3), ld_y=64)
        a.update(kw)
        return lib().mx_combine(*a.values(), None)

    def g(**kw):
        a = dict(dy=at(0), dtype=1, T=10, N=64, ld=64, rows=at(1), ld_r=64, slot=at(2), weight=at(3), src=at(4), k=2,
                 M=20, drows=at(5), ld_d=64, dw=at(6))
        a.update(kw)
        return lib().mx_combine_grad(*a.values(), None)

    for n in ("rows", "slot", "y"):
        assert c(**{n: None}) == NULL, n
    for n in ("dy", "rows", "slot", "src", "drows"):
        assert g(**{n: None}) == NULL, n
    assert c(dtype=9) == DTYPE and g(dtype=9) == DTYPE
    assert c(k=65) == SHAPE and g(k=0) == SHAPE and g(T=-1) == SHAPE
    assert c(ld=63) == STRIDE and c(ld_y=63) == STRIDE and g(ld=63) == STRIDE and g(ld_r=63) == STRIDE
    assert g(ld_d=63) == STRIDE
    assert c(weight=at(2) + 2) == ALIGN and g(dw=at(6) + 1) == ALIGN
    assert c(y=at(0)) == OVERLAP and c(y=at(2)) == OVERLAP
    assert g(drows=at(1)) == OVERLAP and g(dw=at(5)) == OVERLAP and g(dw=at(3)) == OVERLAP
    assert c(T=0, slot=None, y=None) == 0


def test_binding_refuses_host_tensors():
    z = torch.zeros((4, 8))
    i = torch.zeros((4, 2), dtype=torch.int32)
    m = torch.zeros(8, dtype=torch.int32)
    q, s = torch.zeros((4, 8), dtype=torch.int8), torch.zeros(4)
    for f in (lambda: mxq.mx_route(z, 2), lambda: mxq.mx_dispatch(z, i, m), lambda: mxq.mx_dispatch_i8(z, i, m),
              lambda: mxq.i8_quantize_rows(z), lambda: mxq.i8_gemm_nt(q, s, q, s), lambda: mxq.i8_linear(z, q, s),
              lambda: mxq.i8_grouped_gemm_rows(q, s, q[None], s[None], m[:1]), lambda: mxq.mx_combine(z, i),
              lambda: mxq.mx_combine_grad(z, z, i, None, m), lambda: mxq.mx_routing(4, 8, 2, device="cpu"),
              lambda: mxq.mx_routing(4, 8, 9)):
        with pytest.raises(ValueError):
            f()


@pytest.mark.parametrize("normalize", [True, False])
def test_oracle_gradient_against_differences(normalize):
    """The oracle's gradient of <dweight, weight> + dloss loss, picks held."""
    g = np.random.default_rng(5)
    T, E, k = 7, 9, 3
    z = g.normal(size=(T, E))
    z[2, [1, 4]] = -np.inf
    z[3, 1:] = -np.inf
    valid = np.array([1, 1, 1, 1, 0, 1, 1], bool)
    dw, dl = g.normal(size=(T, k)), 0.7
    M = ro.rows_needed(T, E, k, 1)
    r = ro.route(z, valid, k, normalize, 1, M)
    d, _ = ro.route_grad(z, r, k, normalize, dw, dl)

    def f(z):
        q = ro.route(z, valid, k, normalize, 1, M)
        assert (q["idx"] == r["idx"]).all()
        return float((q["weight"] * dw).sum() + dl * q["loss"])

    h = 1e-5
    for t in range(T):
        for e in range(E):
            if not np.isfinite(z[t, e]):
                assert d[t, e] == 0
                continue
            a, b = z.copy(), z.copy()
            a[t, e] += h
            b[t, e] -= h
            assert abs((f(a) - f(b)) / (2 * h) - d[t, e]) < 1e-8, (t, e)
