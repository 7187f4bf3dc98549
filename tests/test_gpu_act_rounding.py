"""GPU tests of bf16 results of products with an epilogue: they are the fp32
formula's values, rounded once.  (The wider bounds that act_oracle has for bf16,
`brief`, are of a formula of fewer operations that results had before.)"""
import pytest
import torch

import act_oracle as ao
import mx9_dual_axis_amd as mxq
from helpers import require_gpu, say
from test_gpu_act import Operand, small_scales
from test_gpu_routed_forms import DEV, codes, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(request):
    require_gpu()
    say(request.node.name)


def rounded(v):
    return v.float().bfloat16().double()


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", ao.ACTS)
def test_values(act, gated):
    """No contraction: the bias alone.  What a value within fp32's error (its
    rounding to fp32 here is one more u) may round to lies between what the ends
    of that error round to."""
    g = gen(51)
    n = 1 << 19
    x = torch.cat([torch.rand(n, generator=g, device=DEV) * 28 - 14, torch.randn(n, generator=g, device=DEV),
                   (torch.rand(n, generator=g, device=DEV) * 80 - 70).exp2() * (torch.randint(0, 2, (n,), generator=g, device=DEV) * 2 - 1),
                   torch.rand(n, generator=g, device=DEV) * 180 - 90])
    x = torch.where(x.abs() > 3e4, 1.0, x)
    bias = torch.cat([x, torch.randn(4 * n, generator=g, device=DEV)]) if gated else x
    W = bias.numel()
    got = mxq.i8_linear_act(torch.empty((1, 0), dtype=torch.bfloat16, device=DEV), torch.empty((W, 0), dtype=torch.int8, device=DEV),
                            torch.ones(W, device=DEV), bias, act, gated)
    want, err = ao.epilogue(bias.double()[None], torch.zeros((1, W), dtype=torch.float64, device=DEV), act, gated)
    err = err + ao.U * (want.abs() + err)
    bad = ~((rounded(want - err) <= got.double()) & (got.double() <= rounded(want + err)))
    assert not bad.any(), (int(bad.sum()), bias[bad[0].nonzero()[0, 0]].item())


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,W,K", [(1, 4096, 512), (13, 700, 1040), (60, 600, 333), (700, 2040, 240), (2000, 4040, 240)])
def test_i8_rounds_the_fp32_result(M, W, K, gated):
    g = gen(M)
    a, b, sa, sb = codes((M, K), g), codes((W, K), g), small_scales(M, K, g), small_scales(W, 1, g)
    bias = torch.randn(W, generator=g, device=DEV)
    res = torch.randn((M, W // 2 if gated else W), generator=g, device=DEV).bfloat16()
    for act in ao.ACTS:
        for r in (None, res):
            one = mxq.i8_gemm_nt_act(a, sa, b, sb, bias, act, gated, r)
            two = mxq.i8_gemm_nt_act(a, sa, b, sb, bias, act, gated, None if r is None else r.float(), out_dtype=torch.float32)
            assert torch.equal(one, two.bfloat16()), (act, r is None)


@pytest.mark.parametrize("form", ["rows", "odd"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,N,K", [(128, 128, 128), (256, 384, 1024), (2048, 1152, 384), (4224, 3968, 128)])
def test_mx_rounds_the_fp32_result(M, N, K, gated, form):
    g = gen(M + N)
    W = 2 * N if gated else N
    A, B = Operand((M, K), g, K), Operand((W, K), g, K)
    bias = torch.randn(W, generator=g, device=DEV)
    res = torch.randn((M, N), generator=g, device=DEV).bfloat16()
    for act in ao.ACTS:
        for r in (None, res):
            ops = (A.q, A.scales(form), B.q, B.scales(form), bias, act, gated)
            one = mxq.mx_gemm_nt_act(*ops, r)
            two = mxq.mx_gemm_nt_act(*ops, None if r is None else r.float(), out_dtype=torch.float32)
            assert torch.equal(one, two.bfloat16()), (act, r is None)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("sizes,N,K", [([128, 0, 256, 128], 256, 512), ([1280, 0, 128, 768], 2048, 256), ([128] * 20 + [0] * 4, 2048, 256)])
@pytest.mark.parametrize("act", ao.ACTS)
def test_by_expert_rounds_the_fp32_result(sizes, N, K, act, gated):
    """MXFP8 and 8-bit, every activation by expert, against binary64 too."""
    g = gen(sum(sizes) + N)
    G, W, M = len(sizes), 2 * N if gated else N, sum(sizes) + 128
    ends = torch.tensor(sizes).cumsum(0)
    offs = ends.int().to(DEV)
    A, B = Operand((M, K), g, K), Operand((G, W, K), g, K)
    bias = torch.randn((G, W), generator=g, device=DEV)
    ops = (A.q, A.s, B.q, B.s, offs, bias, act, gated)
    two, pre = mxq.mx_grouped_gemm_rows_act(*ops, out_dtype=torch.float32, pre=True)
    assert torch.equal(mxq.mx_grouped_gemm_rows_act(*ops), two.bfloat16())
    r0 = 0
    for e, r1 in enumerate(ends.tolist()):
        if r1 > r0:
            x = A.v[r0:r1] @ B.v[e].t().contiguous() + bias[e].double()
            ex = ao.U * x.abs()                                    # test_gpu_act: the bias's addition alone
            assert ((pre[r0:r1].double() - x).abs() <= ex).all(), e
            want, err = ao.epilogue(x, ex, act, gated)
            assert ((two[r0:r1].double() - want).abs() <= err + ao.U * (want.abs() + err)).all(), e
        r0 = r1
    a, sa = codes((M, K), g), small_scales(M, K, g)
    b, sb = codes((G, W, K), g), small_scales(G * W, 1, g).view(G, W)
    ops = (a, sa, b, sb, offs, bias, act, gated)
    assert torch.equal(mxq.i8_grouped_gemm_rows_act(*ops), mxq.i8_grouped_gemm_rows_act(*ops, out_dtype=torch.float32).bfloat16())


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K", [512, 333])
def test_i8_rows_do_not_depend_on_their_batch(K, dtype, gated, biased):
    """With a residual, through forms that add it in different places."""
    g = gen(K + 57)
    M, N = 3000, 333
    W = 2 * N if gated else N
    x, b, sb = torch.randn((M, K), generator=g, device=DEV).to(dtype), codes((W, K), g), small_scales(W, K, g)
    bias = torch.randn(W, generator=g, device=DEV) if biased else None
    res = torch.randn((M, N), generator=g, device=DEV).to(dtype)
    for act in ao.ACTS:
        whole = mxq.i8_linear_act(x, b, sb, bias, act, gated, res)
        for m in (1, 16, 17, 65, 300):
            assert torch.equal(mxq.i8_linear_act(x[:m], b, sb, bias, act, gated, res[:m]), whole[:m]), (act, m)
