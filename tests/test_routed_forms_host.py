"""CPU-only: the rule that chooses the form of an 8-bit product, compiled for the
host from the kernels' own header.  The GPU tests' shapes take the form that
they are listed with, and the lists leave out none that the rule can give."""
import ctypes
import os
import random
import subprocess

import pytest

import routed_shapes as rs

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
KINDS = ("split", "staged", "ring", "pipe")
PIECES, BYTES, FAR = 0, 1, 2


@pytest.fixture(scope="module")
def form(tmp_path_factory):
    d = tmp_path_factory.mktemp("forms")
    (d / "forms.cpp").write_text("""
#include "i8_forms.h"
extern "C" void form(int64_t M, int64_t N, int64_t K, int32_t groups, int32_t rows, int32_t* out) {
    const mxq::Form f = mxq::choose(M, N, K, groups > 0, groups > 0 ? groups : 1, static_cast<mxq::Rows>(rows));
    out[0] = int32_t(f.kind);
    out[1] = f.ms;
    out[2] = f.ns;
}
""")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "mx9_dual_axis_amd", "csrc"), str(d / "forms.cpp"), "-o", str(d / "forms.so")],
                   check=True)
    f = ctypes.CDLL(str(d / "forms.so")).form
    f.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int32] * 2 + [ctypes.c_void_p]
    f.restype = None

    def ask(M, N, K, rows, groups=0):
        out = (ctypes.c_int32 * 3)()
        f(M, N, K, groups, rows, out)
        return KINDS[out[0]], out[1], out[2]

    return ask


def grouped(form, case, rows):
    sizes, N, K = case
    return form(sum(sizes) + rs.TAIL, N, K, rows, len(sizes))


def test_the_listed_shapes_take_the_listed_forms(form):
    for shape, want in rs.DENSE:
        assert form(*shape, BYTES) == want, shape
    for shape, want in rs.FAR:
        assert form(*shape, FAR) == want, shape
    for shape, want in rs.DENSE_PIECES:
        assert form(*shape, PIECES) == want, shape
    for case, want in rs.GROUPS:
        assert grouped(form, case, BYTES) == want, case
    for case, want in rs.GROUP_PIECES:
        assert grouped(form, case, PIECES) == want, case


def test_the_lists_hold_every_form(form):
    g = random.Random(0)
    size = lambda top: int(2 ** g.uniform(0, top))  # noqa: E731
    for listed, rows, by_expert in ((rs.DENSE, BYTES, False), (rs.FAR, FAR, False), (rs.DENSE_PIECES, PIECES, False),
                                    (rs.GROUPS, BYTES, True), (rs.GROUP_PIECES, PIECES, True)):
        given = {form(size(15), size(15), size(14), rows, size(9) if by_expert else 0) for _ in range(20000)}
        assert given == {f for _, f in listed}, (rows, by_expert)
