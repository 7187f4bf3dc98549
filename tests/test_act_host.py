"""CPU-only checks of the epilogue part of the C ABI: declared functions are
exported, arguments are refused on the host, the forms of gated products, and
the binary64 slopes against differences of the activations."""
import os
import re

import pytest
import torch

import act_oracle as ao
import mx9_dual_axis_amd as mxq
import routed_shapes as rs
from mx9_dual_axis_amd import act as binding
from test_routed_forms_host import BYTES, PIECES, form, grouped  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20           # never dereferenced: every call below is refused or empty
NULL, DTYPE, MODE, SHAPE, STRIDE, ALIGN, OVERLAP = 1, 2, 4, 5, 6, 7, 8
F32, BF16 = 0, 1


def at(i):
    return FAKE * (16 + 16 * i)


def lib():
    return binding._L()


def test_every_declared_function_is_exported_and_in_the_package():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "mxq_act.h")).read(), flags=re.S)
    names = re.findall(r"^\s*(?:int|int64_t)\s+(\w+)\s*\(", src, flags=re.M)
    assert len(names) == 9
    for n in names:
        assert hasattr(lib(), n), n
        assert n == "mx_act_grad_workspace" or callable(getattr(mxq, n)), n


def test_the_header_and_the_binding_count_activations_alike():
    src = open(os.path.join(ROOT, "include", "mxq_act.h")).read()
    codes = {k.lower(): int(v) for k, v in re.findall(r"MX_ACT_(\w+) = (\d)", src)}
    assert codes == binding.ACTS and tuple(binding.ACTS) == ao.ACTS


def gemm(**kw):
    a = dict(A=at(0), lda=64, sA=at(1), B=at(2), ldb=64, sB=at(3), M=8, N=32, K=64, act=2, gated=0, bias=at(4), res=at(5),
             ld_res=32, C=at(6), ldc=32, dt=BF16)
    a.update(kw)
    return lib().i8_gemm_nt_act(a["A"], a["lda"], a["sA"], a["B"], a["ldb"], a["sB"], a["M"], a["N"], a["K"], a["act"],
                                a["gated"], a["bias"], a["res"], a["ld_res"], a["C"], a["ldc"], a["dt"], None)


def test_i8_refusals():
    for n in ("A", "sA", "B", "sB", "C"):
        assert gemm(**{n: None}) == NULL, n
    assert gemm(dt=2) == DTYPE
    assert gemm(act=5) == MODE and gemm(act=-1) == MODE
    assert gemm(M=-1) == SHAPE and gemm(K=131072, lda=131072, ldb=131072) == SHAPE and gemm(N=(1 << 30) + 1) == SHAPE
    assert gemm(lda=63) == STRIDE and gemm(ldb=63) == STRIDE and gemm(ldc=31) == STRIDE and gemm(ld_res=31) == STRIDE
    assert gemm(C=at(6) + 1) == ALIGN and gemm(bias=at(4) + 2) == ALIGN and gemm(res=at(5) + 1) == ALIGN
    assert gemm(sA=at(1) + 2) == ALIGN
    for n in ("A", "sA", "B", "sB", "bias"):
        assert gemm(C=at(7), **{n: at(7)}) == OVERLAP, n
    assert gemm(C=at(5) + 2) == OVERLAP                    # the residual, moved
    assert gemm(C=at(5), ldc=40) == OVERLAP                # the residual at another pitch
    # gated: B, its scales and the bias have twice the channels
    end = at(2) + 64 * 64
    assert gemm(gated=1, C=end - 64) == OVERLAP and gemm(gated=0, M=0, C=end - 64) == 0
    assert gemm(gated=1, C=at(3) + 4 * 63) == OVERLAP and gemm(gated=1, C=at(4) + 4 * 63) == OVERLAP
    assert gemm(M=0, A=None, sA=None, B=None, sB=None, C=None, res=None, bias=None) == 0
    assert gemm(N=0, A=None, sA=None, B=None, sB=None, C=None, res=None, bias=None) == 0
    assert gemm(M=0, act=9) == MODE


def linear(**kw):
    a = dict(x=at(0), xd=F32, ld=64, B=at(2), ldb=64, sB=at(3), M=8, N=32, K=64, act=2, gated=0, bias=at(4), res=at(5),
             ld_res=32, C=at(6), ldc=32, dt=BF16, ws=at(7), size=8 * 64 + 32)
    a.update(kw)
    return lib().i8_linear_act(a["x"], a["xd"], a["ld"], a["B"], a["ldb"], a["sB"], a["M"], a["N"], a["K"], a["act"],
                               a["gated"], a["bias"], a["res"], a["ld_res"], a["C"], a["ldc"], a["dt"], a["ws"], a["size"],
                               None)


def test_linear_refusals():
    for n in ("x", "B", "sB", "C", "ws"):
        assert linear(**{n: None}) == NULL, n
    assert linear(xd=3) == DTYPE and linear(dt=3) == DTYPE and linear(act=7) == MODE
    assert linear(size=8 * 64 + 31) == SHAPE
    assert linear(ld=63) == STRIDE and linear(ld_res=3) == STRIDE
    assert linear(ws=at(7) + 8) == ALIGN and linear(x=at(0) + 2) == ALIGN
    for n in ("x", "B", "sB", "bias", "res", "C"):
        assert linear(ws=at(9), **{n: at(9)}) == OVERLAP, n
    assert linear(C=at(0)) == OVERLAP
    assert linear(M=0, x=None, B=None, sB=None, C=None, ws=None, res=None) == 0


def rows(**kw):
    a = dict(A=at(0), lda=64, sA=at(1), B=at(2), ldb=64, bgs=64 * 64, sB=at(3), sgs=64, offs=at(8), G=4, M=8, N=32, K=64,
             act=2, gated=1, bias=at(4), bias_gs=64, C=at(6), ldc=32, dt=BF16)
    a.update(kw)
    return lib().i8_grouped_gemm_rows_act(a["A"], a["lda"], a["sA"], a["B"], a["ldb"], a["bgs"], a["sB"], a["sgs"],
                                          a["offs"], a["G"], a["M"], a["N"], a["K"], a["act"], a["gated"], a["bias"],
                                          a["bias_gs"], a["C"], a["ldc"], a["dt"], None)


def test_grouped_refusals():
    for n in ("A", "sA", "B", "sB", "C", "offs"):
        assert rows(**{n: None}) == NULL, n
    assert rows(act=5) == MODE and rows(G=0) == SHAPE
    assert rows(bias_gs=-1) == STRIDE and rows(bgs=-1) == STRIDE and rows(sgs=-1) == STRIDE
    assert rows(offs=at(8) + 1) == ALIGN
    assert rows(C=at(4) + 4 * (3 * 64 + 63)) == OVERLAP    # the last expert's bias
    assert rows(C=at(8)) == OVERLAP and rows(C=at(2) + 4 * 4096 - 64) == OVERLAP
    assert rows(M=0) == 0


def mx(**kw):
    a = dict(A=at(0), lda=256, sA=at(1), sars=8, sabs=1, B=at(2), ldb=256, sB=at(3), sbrs=8, sbbs=1, M=128, N=128, K=256,
             act=3, gated=1, bias=at(4), res=at(5), ld_res=128, C=at(6), ldc=128, pre=at(7), ld_pre=256, dt=BF16)
    a.update(kw)
    return lib().mx_gemm_nt_act(a["A"], a["lda"], a["sA"], a["sars"], a["sabs"], a["B"], a["ldb"], a["sB"], a["sbrs"],
                                a["sbbs"], a["M"], a["N"], a["K"], a["act"], a["gated"], a["bias"], a["res"], a["ld_res"],
                                a["C"], a["ldc"], a["pre"], a["ld_pre"], a["dt"], None)


def test_mx_refusals():
    for n in ("A", "sA", "B", "sB", "C"):
        assert mx(**{n: None}) == NULL, n
    assert mx(dt=2) == DTYPE and mx(act=5) == MODE
    assert mx(N=64, ldc=128) == SHAPE and mx(N=192) == SHAPE and mx(M=100) == SHAPE and mx(K=200) == SHAPE
    assert mx(N=-128) == SHAPE and mx(N=1 << 24, ldc=1 << 24) == SHAPE     # 2^25 channels
    assert mx(ldc=127) == STRIDE and mx(ld_pre=255) == STRIDE and mx(ld_res=127) == STRIDE and mx(lda=250) == STRIDE
    assert mx(A=at(0) + 8) == ALIGN and mx(pre=at(7) + 1) == ALIGN and mx(res=at(5) + 1) == ALIGN and mx(bias=at(4) + 1) == ALIGN
    for n in ("A", "sA", "B", "sB", "bias", "C", "res"):
        assert mx(pre=at(9), **{n: at(9)}) == OVERLAP, n
    assert mx(C=at(2) + 256 * 256 - 2) == OVERLAP          # the last channel's codes
    assert mx(C=at(3) + 255 * 8 + 6) == OVERLAP
    assert mx(C=at(5) + 256) == OVERLAP
    assert mx(M=0, A=None, sA=None, B=None, sB=None, C=None, pre=None, res=None, bias=None) == 0


def test_mx_grouped_and_matrix_core_refusals():
    def g(mfma=False, **kw):
        a = dict(A=at(0), sA=at(1), B=at(2), sB=at(3), offs=at(8), G=2, N=128, gated=1, act=2, bias=at(4), bgs=256, C=at(6),
                 pre=at(7), b_gs=256 * 256, s_gs=256 * 8)
        a.update(kw)
        mid = (a["act"], a["gated"], a["bias"], a["bgs"], a["C"], 128, a["pre"], 256, BF16, None)
        if mfma:
            return lib().mx_grouped_gemm_rows_act_mfma(a["A"], 256, a["sA"], a["B"], 256, a["b_gs"], a["sB"], a["s_gs"],
                                                       a["offs"], a["G"], 256, a["N"], 256, *mid)
        return lib().mx_grouped_gemm_rows_act(a["A"], 256, a["sA"], 8, 1, a["B"], 256, a["b_gs"], a["sB"], 8, 1, a["s_gs"],
                                              a["offs"], a["G"], 256, a["N"], 256, *mid)

    for mfma in (False, True):
        for n in ("A", "sA", "B", "sB", "C", "offs"):
            assert g(mfma, **{n: None}) == NULL, n
        assert g(mfma, act=-1) == MODE and g(mfma, G=0) == SHAPE and g(mfma, N=64) == SHAPE
        assert g(mfma, bgs=-1) == STRIDE and g(mfma, b_gs=-1) == STRIDE
        assert g(mfma, offs=at(8) + 2) == ALIGN
        assert g(mfma, C=at(4) + 4 * 511) == OVERLAP and g(mfma, pre=at(8)) == OVERLAP
    assert g(True, sA=at(1) + 4) == ALIGN
    assert lib().mx_gemm_nt_act_mfma(at(0), 256, at(1), at(2), 256, at(3) + 8, 128, 128, 256, 0, 0, None, None, 0, at(6), 128,
                                     None, 0, F32, None) == ALIGN


def grad(**kw):
    a = dict(dy=at(0), ldy=40, pre=at(1), ldp=80, dt=F32, M=50, N=40, act=2, gated=1, offs=None, G=0, d=at(2), ldd=80,
             db=at(3), ws=at(4), size=1 << 20)
    a.update(kw)
    return lib().mx_act_grad(a["dy"], a["ldy"], a["pre"], a["ldp"], a["dt"], a["M"], a["N"], a["act"], a["gated"], a["offs"],
                             a["G"], a["d"], a["ldd"], a["db"], a["ws"], a["size"], None)


def test_gradient_refusals():
    for n in ("dy", "pre", "d", "ws"):
        assert grad(**{n: None}) == NULL, n
    assert grad(dt=2) == DTYPE and grad(act=5) == MODE
    assert grad(M=-1) == SHAPE and grad(offs=at(5), G=0) == SHAPE and grad(offs=at(5), G=65536) == SHAPE and grad(size=100) == SHAPE
    assert grad(N=(1 << 30) + 1) == SHAPE and grad(N=65535 * 128 + 1, ldy=1 << 30, ldp=1 << 30, ldd=1 << 30) == SHAPE
    assert grad(ldy=39) == STRIDE and grad(ldp=79) == STRIDE and grad(ldd=79) == STRIDE
    assert grad(dy=at(0) + 2) == ALIGN and grad(db=at(3) + 1) == ALIGN and grad(offs=at(5) + 1, G=2) == ALIGN
    assert grad(d=at(1)) == OVERLAP and grad(d=at(0)) == OVERLAP and grad(db=at(4)) == OVERLAP and grad(ws=at(1)) == OVERLAP
    assert grad(M=0, db=None) == 0 and grad(N=0) == 0
    w = lib().mx_act_grad_workspace
    assert w(-1, 4, F32, 0, 0) == -1 and w(4, 4, 2, 0, 0) == -1 and w(4, 4, F32, 0, 65536) == -1 and w(4, 4, F32, 0, -1) == -1
    assert w(0, 4, F32, 0, 3) == 0
    # every group and the tail may end in a row tile of its own
    assert w(100, 64, BF16, 1, 7) >= (100 // 256 + 8) * 128 * 4


def test_gated_products_take_every_tiled_form(form):  # noqa: F811
    """The shapes of the GPU tests, halved and doubled again: no tile that the
    listed shapes take is left out."""
    pair = lambda n: 2 * (n // 2)  # noqa: E731
    for cases, rows_, by in ((rs.DENSE, BYTES, False), (rs.DENSE_PIECES, PIECES, False), (rs.GROUPS, BYTES, True),
                             (rs.GROUP_PIECES, PIECES, True)):
        if by:
            took = {grouped(form, (c[0], pair(c[1]), c[2]), rows_) for c, _ in cases}
        else:
            took = {form(c[0], pair(c[1]), c[2], rows_) for c, _ in cases}
        assert took == {f for _, f in cases}


@pytest.mark.parametrize("name", ao.ACTS)
def test_slopes_are_those_of_the_activations(name):
    x = torch.linspace(-9, 9, 3601, dtype=torch.float64) + 0.0003
    h = 1e-5
    want = (ao.act(x + h, name) - ao.act(x - h, name)) / (2 * h)
    s, _ = ao.slope(x, name)
    assert (s - want).abs().max() < 1e-8
    gate, up = x[:3600:2][None], x[1:3600:2][None]
    pre, dy = torch.cat([gate, up], 1), torch.cos(gate)
    d, _ = ao.grad(dy, pre, name, True)
    f = lambda p: (ao.epilogue(p, torch.zeros_like(p), name, True)[0] * dy).sum()  # noqa: E731
    for i in (0, 100, 901, 1799, 1800, 2500, 3599):
        e = torch.zeros_like(pre)
        e[0, i] = h
        assert abs(float((f(pre + e) - f(pre - e)) / (2 * h) - d[0, i])) < 1e-5
