"""GPU tests of the 8-bit products in every form of their kernels, at shapes that
are known to take it (test_routed_forms_host asks the rule itself).  Tolerances
are those of the operations: 4 u of the magnitudes and 2^-8 |C| in bf16."""
import numpy as np
import pytest
import torch

import mx9_dual_axis_amd as mxq
import routed_oracle as ro
import routed_shapes as rs
from helpers import require_gpu, say
from test_gpu_routed_forms import DEV, DT, at_any_byte, codes, gen, near, plain, scales

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(request):
    require_gpu()
    say(request.node.name)


def name(case):
    if isinstance(case, bool):
        return "pieces" if case else "bytes"
    return "-".join(str(x) if isinstance(x, (int, str)) else f"{len(x)}groups" for x in case)


def check_dense(A, B, a, b, sa, sb, out, bias):
    M, N = a.shape[0], b.shape[0]
    want, mag = plain(a, sa, b, sb, bias)
    buf = torch.full((M, N + 3), 99, dtype=DT[out], device=DEV)
    near(mxq.i8_gemm_nt(A, sa, B, sb, bias, out=buf[:, :N]), want, mag, DT[out], "pitched result")
    assert (buf[:, N:] == 99).all()
    near(mxq.i8_gemm_nt(A, sa, B, sb, bias, out_dtype=DT[out]), want, mag, DT[out], "whole result")


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("shape,pieces", [(s, False) for s, _ in rs.DENSE] + [(s, True) for s, _ in rs.DENSE_PIECES],
                         ids=name)
def test_dense(shape, pieces, out):
    M, N, K = shape
    g = gen(M + N + K)
    a, b, sa, sb = codes((M, K), g), codes((N, K), g), scales(M, g), scales(N, g)
    bias = torch.randn(N, generator=g, device=DEV) * 50
    A, B = (a, b) if pieces else (at_any_byte(a), at_any_byte(b))
    check_dense(A, B, a, b, sa, sb, out, bias)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [s for s, _ in rs.FAR], ids=name)
def test_rows_far_apart(shape, out):
    M, N, K = shape
    g = gen(M + N + K)
    a, b, sa, sb = codes((M, K), g), codes((N, K), g), scales(M, g), scales(N, g)
    bias = torch.randn(N, generator=g, device=DEV) * 50
    few, pitch = min(M, N), 2 ** 23 + 16
    buf = torch.empty(few * pitch, dtype=torch.int8, device=DEV)
    v = buf.as_strided((few, K), (pitch, 1))
    v.copy_(a if M < N else b)
    A, B = (v, b) if M < N else (a, v)
    check_dense(A, B, a, b, sa, sb, out, bias)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("case,pieces", [(c, False) for c, _ in rs.GROUPS] + [(c, True) for c, _ in rs.GROUP_PIECES],
                         ids=name)
def test_by_expert(case, pieces, out):
    sizes, N, K = case
    g = gen(len(sizes) + N + K)
    M, G = sum(sizes) + rs.TAIL, len(sizes)
    a, b, sa, sb = codes((M, K), g), codes((G, N, K), g), scales(M, g), scales((G, N), g)
    offs = np.cumsum(sizes)
    want, mag = torch.zeros((M, N), dtype=torch.float64, device=DEV), torch.zeros((M, N), dtype=torch.float64, device=DEV)
    for e, (r0, r1) in enumerate(ro.group_ranges(offs, M)):
        want[r0:r1], mag[r0:r1] = plain(a[r0:r1], sa[r0:r1], b[e], sb[e])
    sa[offs[-1]:] = float("nan")                          # the tail is no group's
    od = torch.from_numpy(offs.astype(np.int32)).to(DEV)
    A, B = (a, b) if pieces else (at_any_byte(a), at_any_byte(b))
    buf = torch.full((M, N + 3), 99, dtype=DT[out], device=DEV)
    near(mxq.i8_grouped_gemm_rows(A, sa, B, sb, od, out=buf[:, :N]), want, mag, DT[out], "pitched result")
    assert (buf[:, N:] == 99).all()
    near(mxq.i8_grouped_gemm_rows(A, sa, B, sb, od, out_dtype=DT[out]), want, mag, DT[out], "whole result")
