"""GPU tests of the products with an epilogue and of its gradient, against
binary64 (act_oracle, which derives the errors of the activations).

  * 8-bit: the sum is exact; its conversion, two products and the bias add round
    once each, 4 u of the magnitudes.
  * MXFP8: operands whose products the matrix cores add without loss (E4M3 values
    0.25 .. 3.75, scales constant along the contraction) give x up to the
    bias's addition, u (|x|); others within (2^-10 + (K + 2) 2^-24) of the
    magnitudes, as the contraction itself.
  * a result rounds once more: 2^-8 of it in bf16.
  * sums of dpre: a thread adds 32 rows at most, then 8, a segment of the row
    tiles and 16 segments.
"""
import numpy as np
import pytest
import torch

import act_oracle as ao
import mx9_dual_axis_amd as mxq
import routed_oracle as ro
import routed_shapes as rs
from helpers import require_gpu, say
from test_gpu_routed_forms import DEV, DT, at_any_byte, codes, gen, scales

pytestmark = pytest.mark.gpu
U = ao.U


@pytest.fixture(autouse=True)
def _gpu(request):
    require_gpu()
    say(request.node.name)


def near(got, want, err, what):
    e = err + (2.0 ** -8 * (want.abs() + err) if got.dtype == torch.bfloat16 else 0)
    g = got.double()
    bad = ~((g - want).abs() <= e) & ~(g.isnan() & want.isnan())
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        pytest.fail(f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound; first {i}: got {g[i].item()!r} "
                    f"want {want[i].item()!r} bound {e[i].item()!r}")


def sums8(a, sa, b, sb, bias):
    """(x, its error) of an 8-bit product."""
    x = (a.double() @ b.double().t().contiguous()) * sa.double()[:, None] * sb.double()
    mag = x.abs()
    if bias is not None:
        x, mag = x + bias.double(), mag + bias.double().abs()
    return x, 4 * U * mag


def name(case):
    if isinstance(case, bool):
        return "pieces" if case else "bytes"
    if isinstance(case, tuple):
        return "-".join(str(x) if isinstance(x, (int, str)) else f"{len(x)}groups" for x in case)
    return None


def small_scales(n, K, g):
    """Scales that put sums of K codes around 1, where activations bend."""
    return torch.exp2(torch.rand(n, generator=g, device=DEV) * 4 - 2) / (70 * K ** 0.5)


def epilogue_case(i):
    return ao.ACTS[i % 5], i % 3 != 0, i % 2 == 0        # activation, bias, residual


# ----------------------------------------------------------- 8-bit products
DENSE = [(s, False) for s, _ in rs.DENSE] + [(s, True) for s, _ in rs.DENSE_PIECES]
GROUPS = [(c, False) for c, _ in rs.GROUPS] + [(c, True) for c, _ in rs.GROUP_PIECES]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("i", range(len(DENSE)), ids=lambda i: name(DENSE[i][0]) + "-" + name(DENSE[i][1]))
def test_dense_in_every_form(i, out, gated):
    (M, W, K), pieces = DENSE[i]
    N = W // 2 if gated else W
    W = 2 * N if gated else N
    act, has_bias, has_res = epilogue_case(i + gated)
    g = gen(M + W + K)
    a, b, sa, sb = codes((M, K), g), codes((W, K), g), small_scales(M, K, g), small_scales(W, 1, g)
    bias = torch.randn(W, generator=g, device=DEV) if has_bias else None
    buf = torch.full((M, N + 3), 99.0, dtype=DT[out], device=DEV)
    wide = torch.randn((M, N + 5), generator=g, device=DEV).to(DT[out])
    res = wide[:, 2:N + 2] if has_res else None
    x, ex = sums8(a, sa, b, sb, bias)
    want, err = ao.epilogue(x, ex, act, gated, None if res is None else res.double(), out == "bf16")
    A, B = (a, b) if pieces else (at_any_byte(a), at_any_byte(b))
    mxq.i8_gemm_nt_act(A, sa, B, sb, bias, act, gated, res, out=buf[:, :N])
    near(buf[:, :N], want, err, "pitched result")
    assert (buf[:, N:] == 99).all()
    whole = None if res is None else res.contiguous()
    near(mxq.i8_gemm_nt_act(A, sa, B, sb, bias, act, gated, whole, out_dtype=DT[out]), want, err, "whole result")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("i", range(len(GROUPS)), ids=lambda i: name(GROUPS[i][0]) + "-" + name(GROUPS[i][1]))
def test_by_expert_in_every_form(i, out, gated):
    (sizes, W, K), pieces = GROUPS[i]
    N = W // 2 if gated else W
    W = 2 * N if gated else N
    act, has_bias, _ = epilogue_case(i + gated)
    g = gen(len(sizes) + W + K)
    M, G = sum(sizes) + rs.TAIL, len(sizes)
    a, b, sa, sb = codes((M, K), g), codes((G, W, K), g), small_scales(M, K, g), small_scales(G * W, 1, g).view(G, W)
    bias = torch.randn((G + 1, W + 3), generator=g, device=DEV)[:, 1:W + 1] if has_bias else None
    offs = np.cumsum(sizes)
    want, err = (torch.zeros((M, N), dtype=torch.float64, device=DEV) for _ in range(2))
    for e, (r0, r1) in enumerate(ro.group_ranges(offs, M)):
        x, ex = sums8(a[r0:r1], sa[r0:r1], b[e], sb[e], None if bias is None else bias[e])
        want[r0:r1], err[r0:r1] = ao.epilogue(x, ex, act, gated, None, out == "bf16")
    sa[offs[-1]:] = float("nan")                          # the tail is no group's
    od = torch.from_numpy(offs.astype(np.int32)).to(DEV)
    A, B = (a, b) if pieces else (at_any_byte(a), at_any_byte(b))
    buf = torch.full((M, N + 3), 99.0, dtype=DT[out], device=DEV)
    mxq.i8_grouped_gemm_rows_act(A, sa, B, sb, od, bias, act, gated, out=buf[:, :N])
    near(buf[:, :N], want, err, "pitched result")
    assert (buf[:, N:] == 99).all()
    near(mxq.i8_grouped_gemm_rows_act(A, sa, B, sb, od, bias, act, gated, out_dtype=DT[out]), want, err, "whole result")


# Activations quantized by the ring, by the split form, by a kernel before.
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 7168, 4096), (1, 4096, 512), (1, 16, 8192), (3, 8201, 1040), (16, 40, 256),
                                   (16, 70, 528), (17, 40, 15), (77, 500, 1111), (40, 333, 2049), (300, 800, 600),
                                   (1000, 1001, 240)])
def test_linear(M, N, K, dtype, gated):
    g = gen(M + N + K)
    W = 2 * N if gated else N
    x = torch.randn((M, K), generator=g, device=DEV).to(DT[dtype])
    b, sb = codes((W, K), g), small_scales(W, K, g)
    bias = torch.randn(W, generator=g, device=DEV)
    q, s = mxq.i8_quantize_rows(x)
    for i, act in enumerate(ao.ACTS):
        res = torch.randn((M, N), generator=g, device=DEV).to(DT[dtype]) if i % 2 else None
        bi = bias if i != 2 else None
        of = (*sums8(q, s, b, sb, bi), act, gated, None if res is None else res.double())
        want, err = ao.epilogue(*of, dtype == "bf16")
        near(mxq.i8_linear_act(x, b, sb, bi, act, gated, res), want, err, act)
        got = mxq.i8_linear_act(x, b, sb, bi, act, gated, None if res is None else res.float(), out_dtype=torch.float32)
        near(got, *ao.epilogue(*of), f"{act}, fp32")


def test_without_an_epilogue_the_bits_are_those_of_the_product():
    g = gen(3)
    for M, N, K in [(1, 4096, 512), (13, 700, 1040), (60, 600, 333), (700, 2040, 240)]:
        x, b, sb = torch.randn((M, K), generator=g, device=DEV), codes((N, K), g), small_scales(N, K, g)
        bias = torch.randn(N, generator=g, device=DEV)
        for bi in (None, bias):
            assert torch.equal(mxq.i8_linear_act(x, b, sb, bi), mxq.i8_linear(x, b, sb, bi))


def test_the_same_rows_give_the_same_bits_in_any_batch():
    """A token's results do not depend on what it is batched with, though the
    forms differ."""
    g = gen(4)
    x, b = torch.randn((300, 512), generator=g, device=DEV), codes((2 * 333, 512), g)
    sb, bias = small_scales(666, 512, g), torch.randn(666, generator=g, device=DEV)
    for act in ao.ACTS:
        all_ = mxq.i8_linear_act(x, b, sb, bias, act, True)
        for M in (1, 16, 17, 65):
            assert torch.equal(mxq.i8_linear_act(x[:M], b, sb, bias, act, True), all_[:M]), (act, M)


@pytest.mark.parametrize("M,N,K", [(1, 40, 64), (5, 8200, 256), (60, 600, 333), (700, 2040, 240), (2000, 4040, 240)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_residual_in_place(M, N, K, dtype):
    g = gen(M)
    x, b, sb = torch.randn((M, K), generator=g, device=DEV).to(DT[dtype]), codes((N, K), g), small_scales(N, K, g)
    res = torch.randn((M, N), generator=g, device=DEV).to(DT[dtype])
    want = mxq.i8_linear_act(x, b, sb, None, "gelu", False, res)
    y = res.clone()
    got = mxq.i8_linear_act(x, b, sb, None, "gelu", False, y, out=y)
    assert got is y and torch.equal(y, want)


def test_values_that_are_not_finite():
    """A NaN or infinity of a row's scale, a channel's bias or the residual stays
    in its row, its channel, its element."""
    g = gen(6)
    for M, K in ((3, 64), (70, 333), (300, 240)):
        N = 500
        a, b, sa, sb = codes((M, K), g), codes((N, K), g), small_scales(M, K, g), small_scales(N, 1, g)
        bias, res = torch.randn(N, generator=g, device=DEV), torch.randn((M, N), generator=g, device=DEV)
        sa[1], bias[7], bias[8], bias[9], res[0, 5] = float("nan"), float("inf"), -float("inf"), float("nan"), float("nan")
        for act in ao.ACTS:
            y = mxq.i8_gemm_nt_act(a, sa, b, sb, bias, act, False, res, out_dtype=torch.float32)
            assert y[1].isnan().all() and y[:, 9].isnan().all() and y[0, 5].isnan()
            assert (y[0, 7] == float("inf")) and (act != "relu" or y[0, 8] == res[0, 8])
            ok = torch.ones_like(y, dtype=torch.bool)
            ok[1], ok[:, 7:10], ok[0, 5] = False, False, False
            assert y[ok].isfinite().all(), act


def test_empty():
    g = gen(7)
    b, sb, bias = codes((40, 32), g), small_scales(40, 32, g), torch.randn(40, generator=g, device=DEV)
    x = torch.randn((0, 32), generator=g, device=DEV)
    assert mxq.i8_linear_act(x, b, sb, act="silu", gated=True).shape == (0, 20)
    assert mxq.i8_linear_act(torch.randn((3, 32), device=DEV), b[:0], sb[:0], act="silu", gated=True).shape == (3, 0)
    # no contraction: the bias alone
    y = mxq.i8_linear_act(torch.empty((3, 0), device=DEV), b[:, :0], sb, bias, "silu")
    want, err = ao.epilogue(bias.double().expand(3, 40), torch.zeros((3, 40), dtype=torch.float64, device=DEV), "silu", False)
    near(y, want, err, "no contraction")


# ------------------------------------------------------------ MXFP8 products
def narrow(shape, g):
    """E4M3 values 0.25 .. 3.75 of either sign, as codes and in binary64."""
    e = torch.randint(6, 9, shape, generator=g, device=DEV)
    q = (torch.randint(0, 2, shape, generator=g, device=DEV) << 7) | (e << 3) | torch.randint(0, 8, shape, generator=g,
                                                                                             device=DEV)
    q = q.to(torch.uint8)
    return q, q.view(torch.float8_e4m3fn).double()


class Operand:
    """Codes [.., rows, K] and scales in each layout."""

    def __init__(self, shape, g, K):
        self.q, v = narrow(shape, g)
        s = torch.randint(119, 124, (*shape[:-1], 1), generator=g, device=DEV)      # 2^-8 .. 2^-4
        self.s = s.expand(*shape[:-1], K // 32).to(torch.uint8).contiguous()
        self.v = v * torch.exp2(s.double() - 127)

    def scales(self, form):
        if form == "rows":
            return self.s
        if form == "odd":                                      # neither adjacent blocks nor adjacent rows
            w = self.s.repeat_interleave(3, dim=-1)
            return w[..., ::3]
        if form == "blocks":
            return self.s.transpose(-1, -2).contiguous().transpose(-1, -2)
        if self.s.dim() == 2:
            return mxq.scales_to_mfma(self.s)
        return torch.stack([mxq.scales_to_mfma(x) for x in self.s])


FORMS = ("rows", "blocks", "mfma", "odd")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("out", ["f32", "bf16"])
# Tiles of 64 x 64 whose waves split the contraction (the first four, with fewer
# steps than waves and more), of 128 x 256, of 256 x 256, ragged ones among them.
@pytest.mark.parametrize("M,N,K", [(128, 128, 128), (1920, 5120, 256), (256, 384, 1024), (384, 640, 512), (640, 256, 1152), (2048, 1920, 256),
                                   (2048, 1152, 384), (4224, 3968, 128), (3968, 4224, 256)])
def test_mx_dense(M, N, K, out, gated):
    g = gen(M + N + K)
    W = 2 * N if gated else N
    A, B = Operand((M, K), g, K), Operand((W, K), g, K)
    bias = torch.randn(W, generator=g, device=DEV)
    buf = torch.full((M, N + 3), 99.0, dtype=DT[out], device=DEV)
    kept = torch.full((M, W + 3), 99.0, dtype=DT[out], device=DEV)
    for i, act in enumerate(ao.ACTS):
        form = FORMS[(i + gated + M // 128) % 4]
        bi = bias if i % 3 else None
        res = torch.randn((M, N + 1), generator=g, device=DEV).to(DT[out])[:, 1:] if i % 2 else None
        x = A.v @ B.v.t().contiguous() + (0 if bi is None else bi.double())
        ex = U * x.abs()
        want, err = ao.epilogue(x, ex, act, gated, None if res is None else res.double(), out == "bf16")
        call = mxq.mx_gemm_nt_act_mfma if form == "mfma" else mxq.mx_gemm_nt_act
        ops = (A.q, A.scales(form), B.q, B.scales(form))
        call(*ops, bi, act, gated, res, out=buf[:, :N], pre=kept[:, :W])
        near(buf[:, :N], want, err, f"{act} {form}: y")
        near(kept[:, :W], x, ex, f"{act} {form}: pre")
        assert (buf[:, N:] == 99).all() and (kept[:, W:] == 99).all()
        y, pre = call(*ops, bi, act, gated, None if res is None else res.contiguous(), out_dtype=DT[out], pre=True)
        assert torch.equal(y, buf[:, :N]) and torch.equal(pre, kept[:, :W]), f"{act} {form}: whole rows"
        assert torch.equal(call(*ops, bi, act, gated, res, out_dtype=DT[out]), y), f"{act} {form}: without pre"


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("sizes,tail,N,K", [([128, 0, 256, 128], 128, 256, 512), ([0, 0, 384], 0, 128, 256),
                                            ([128] * 5 + [640], 256, 384, 1152),
                                            ([1280, 0, 128, 768], 640, 2048, 256), ([128, 256] * 8, 128, 1024, 384),
                                            ([128] * 20 + [0] * 4, 128, 2048, 256), ([0, 384] * 35 + [256], 384, 640, 256),
                                            ([640, 0, 1152, 128], 128, 3200, 128)])
def test_mx_by_expert(sizes, tail, N, K, out, gated, form):
    g = gen(sum(sizes) + N)
    M, G, W = sum(sizes) + tail, len(sizes), 2 * N if gated else N
    A, B = Operand((M, K), g, K), Operand((G, W, K), g, K)
    bias = torch.randn((G, W), generator=g, device=DEV)
    ends = np.cumsum(sizes)
    offs = torch.from_numpy(ends.astype(np.int32)).to(DEV)
    x = torch.zeros((M, W), dtype=torch.float64, device=DEV)
    for e, (r0, r1) in enumerate(ro.group_ranges(ends, M)):
        x[r0:r1] = A.v[r0:r1] @ B.v[e].t().contiguous() + bias[e].double()
    want, err = ao.epilogue(x, U * x.abs(), "silu", gated, None, out == "bf16")
    want[ends[-1]:] = 0
    call = mxq.mx_grouped_gemm_rows_act_mfma if form == "mfma" else mxq.mx_grouped_gemm_rows_act
    y, pre = call(A.q, A.scales(form), B.q, B.scales(form), offs, bias, "silu", gated, out_dtype=DT[out], pre=True)
    near(y, want, err, "y")
    near(pre, x, U * x.abs(), "pre")
    assert not y[ends[-1]:].any() and not pre[ends[-1]:].any()


@pytest.mark.parametrize("gated", [False, True])
def test_a_bias_that_experts_share_and_experts_without_rows(gated):
    """70 groups of a stack of 73 experts; the bias by a pitch of 0, by one that
    is wider than its rows, and contiguous: the same bits."""
    g = gen(70 + gated)
    E, G, N, K = 73, 70, 128, 128
    W = 2 * N if gated else N
    sizes = np.array([128 * (e % 3 == 0) for e in range(G)])
    offs = torch.from_numpy(np.cumsum(sizes).astype(np.int32)).to(DEV)
    M = int(sizes.sum()) + 128
    one = torch.randn(W, generator=g, device=DEV)
    wide = torch.full((E, W + 5), float("nan"), device=DEV)
    wide[:, :W] = one
    A, B = Operand((M, K), g, K), Operand((E, W, K), g, K)
    qa, sa = mxq.i8_quantize_rows(torch.randn((M, K), generator=g, device=DEV))
    qb, sb = mxq.i8_quantize_rows(torch.randn((E * W, K), generator=g, device=DEV) * K ** -0.5)
    qb, sb = qb.view(E, W, K), sb.view(E, W)
    calls = (lambda b: mxq.mx_grouped_gemm_rows_act(A.q, A.scales("rows"), B.q, B.scales("rows"), offs, b, "silu", gated),
             lambda b: mxq.i8_grouped_gemm_rows_act(qa, sa, qb, sb, offs, b, "silu", gated))
    for call in calls:
        want = call(one.repeat(E, 1))
        assert want[:M - 128].any(1).all() and not want[M - 128:].any()
        assert torch.equal(call(one.expand(E, W)), want)
        assert torch.equal(call(wide[:, :W]), want)
        assert torch.equal(call(one.repeat(G, 1)), want)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("gated", [False, True])
def test_mx_by_many_experts(gated, form):
    """70 experts whose B exceed the last cache, and 23 of them at a time: the
    same rows give the same bits."""
    g = gen(69 + gated)
    G, W, K = 70, 2048, 2048
    N = W // 2 if gated else W
    sizes = np.array([0, 128, 256, 384, 512, 128, 384] * 10)
    ends = np.cumsum(sizes)
    M = int(ends[-1]) + 256
    A = Operand((M, K), g, K)
    B = Operand((G, W, K), g, K)
    B.v = None
    bias = torch.randn((G, W), generator=g, device=DEV)
    call = mxq.mx_grouped_gemm_rows_act_mfma if form == "mfma" else mxq.mx_grouped_gemm_rows_act
    sA, sB = A.scales(form), B.scales(form)
    offs = torch.from_numpy(ends.astype(np.int32)).to(DEV)
    y, pre = call(A.q, sA, B.q, sB, offs, bias, "gelu", gated, pre=True)
    assert not y[ends[-1]:].any() and not pre[ends[-1]:].any()
    for e0 in range(0, G, 23):
        e1 = min(e0 + 23, G)
        r0, r1 = int(ends[e0] - sizes[e0]), int(ends[e1 - 1])
        rows = A.s[r0:r1]
        part = {"rows": lambda s: s, "odd": lambda s: s.repeat_interleave(3, dim=-1)[..., ::3],
                "blocks": lambda s: s.transpose(-1, -2).contiguous().transpose(-1, -2), "mfma": mxq.scales_to_mfma}[form](rows)
        ye, pe = call(A.q[r0:r1], part, B.q[e0:e1], sB[e0:e1], offs[e0:e1] - r0, bias[e0:e1], "gelu", gated, pre=True)
        assert torch.equal(y[r0:r1], ye) and torch.equal(pre[r0:r1], pe), e0


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("sizes,tail,N,K", [([640, 0, 1152, 128], 384, 3200, 128), ([128] * 20 + [0] * 4, 256, 2048, 256),
                                            ([128, 0, 256], 128, 128, 256)])
def test_mx_by_expert_into_any_rows(sizes, tail, N, K, gated, out):
    """Results and kept sums at any element and pitch: the bits of contiguous
    ones, the tail 0, what surrounds them as it was."""
    g = gen(sum(sizes) + K)
    M, G, W = sum(sizes) + tail, len(sizes), 2 * N if gated else N
    A, B = Operand((M, K), g, K), Operand((G, W, K), g, K)
    bias = torch.randn((G, W), generator=g, device=DEV)
    offs = torch.from_numpy(np.cumsum(sizes).astype(np.int32)).to(DEV)
    ops = (A.q, A.s, B.q, B.s, offs, bias, "gelu_tanh", gated)
    want, kept = mxq.mx_grouped_gemm_rows_act(*ops, out_dtype=DT[out], pre=True)
    assert not want[M - tail:].any() and not kept[M - tail:].any() and want[:M - tail].any(1).all()
    y, pre = (torch.full((M, n + 5), 9.0, dtype=DT[out], device=DEV) for n in (N, W))
    mxq.mx_grouped_gemm_rows_act(*ops, out=y[:, 3:N + 3], pre=pre[:, 1:W + 1])
    assert torch.equal(y[:, 3:N + 3], want) and torch.equal(pre[:, 1:W + 1], kept)
    assert (y[:, :3] == 9).all() and (y[:, N + 3:] == 9).all() and (pre[:, :1] == 9).all() and (pre[:, W + 1:] == 9).all()


@pytest.mark.parametrize("M,N,K", [(2304, 3200, 128), (1280, 3200, 256), (384, 128, 256)])
def test_mx_ends_that_are_none(M, N, K):
    """Ends below 0, past the rows, descending or inside a unit: as the ends
    rounded down to units and clamped to an ascending sequence."""
    g = gen(M)
    bad = np.array([-300, 300, 130, 10 ** 9, 700, -2 ** 31, M + 1, 2 ** 31 - 1])[[0, 1, 2, 4, 5, 3, 6, 7]]
    good = np.maximum.accumulate(np.clip(bad, 0, M) // 128 * 128)
    A, B = Operand((M, K), g, K), Operand((8, N, K), g, K)
    call = lambda e: mxq.mx_grouped_gemm_rows_act(A.q, A.s, B.q, B.s, torch.from_numpy(e.astype(np.int32)).to(DEV), act="silu",  # noqa: E731
                                                  pre=True)
    for n in (5, 8):                                           # with a tail, and the rest to one group
        for a, b in zip(call(bad[:n]), call(good[:n])):
            assert torch.equal(a, b)


def test_mx_without_a_contraction_is_refused():
    """As mx_gemm_nt's: torch's empty operands have no address."""
    q, s = torch.empty((128, 0), dtype=torch.uint8, device=DEV), torch.empty((128, 0), dtype=torch.uint8, device=DEV)
    for call in (mxq.mx_gemm_nt, mxq.mx_gemm_nt_act):
        with pytest.raises(mxq.MXError) as e:
            call(q, s, q, s)
        assert e.value.status == 1


def test_mx_with_ordinary_operands():
    """Codes and scales of the casts, against binary64."""
    g = gen(9)
    M, N, K = 256, 384, 1024
    xa, xb = (torch.randn((r, K), generator=g, device=DEV).bfloat16() for r in (M, 2 * N))
    qa, sa, _, _ = mxq.mx_quantize_2d_dual(xa)
    qb, sb, _, _ = mxq.mx_quantize_2d_dual(xb)
    val = lambda q, s: q.view(torch.float8_e4m3fn).double() * torch.exp2(s.double() - 127).repeat_interleave(32, 1)  # noqa: E731
    va, vb = val(qa, sa), val(qb, sb)
    x = va @ vb.t().contiguous()
    ex = (2.0 ** -10 + (K + 2) * U) * (va.abs() @ vb.abs().t().contiguous())
    y, pre = mxq.mx_gemm_nt_act(qa, sa, qb, sb, act="gelu", gated=True, out_dtype=torch.float32, pre=True)
    near(pre, x, ex, "x")
    near(y, *ao.epilogue(pre.double(), torch.zeros_like(x), "gelu", True), "y from those sums")


# ------------------------------------------------------------------ gradient
def sum_error(d, e, rows, tiles):
    return e.sum(0) + (32 + 8 + 16 + tiles / 16 + 2) * U * (d.abs() + e).sum(0)


@pytest.mark.parametrize("act", ao.ACTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N", [(1, 1), (3, 9), (17, 513), (333, 1111), (4100, 264), (270001, 8)])
def test_gradient(M, N, dtype, gated, act):
    g = gen(M + N)
    W = 2 * N if gated else N
    dy = torch.randn((M, N + 3), generator=g, device=DEV).to(DT[dtype])[:, 1:N + 1]
    pre = (torch.randn((M, W + 5), generator=g, device=DEV) * 3).to(DT[dtype])[:, 3:W + 3]
    d, e = ao.grad(dy.double(), pre.double(), act, gated)
    buf = torch.full((M, W + 3), 99.0, dtype=DT[dtype], device=DEV)
    dbias = torch.full((W,), 99.0, device=DEV)
    mxq.mx_act_grad(dy, pre, act, gated, out=(buf[:, :W], dbias))
    near(buf[:, :W], d, e, "dpre")
    assert (buf[:, W:] == 99).all()
    near(dbias, d.sum(0), sum_error(d, e, M, M / 16 + 1), "dbias")
    dpre, none = mxq.mx_act_grad(dy.contiguous(), pre.contiguous(), act, gated, bias=False)
    assert none is None and torch.equal(dpre, buf[:, :W])


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [8, 301])
@pytest.mark.parametrize("sizes,tail", [([0, 3, 16, 1, 0, 40, 17, 15], 4), ([0, 0], 5), ([1000, 0, 257], 0), ([5] * 130, 7),
                                        ([7, 0, 700] * 50, 100), ([900, 0, 3000], 30)])
def test_gradient_by_expert(sizes, tail, N, dtype, gated):
    g = gen(sum(sizes) + N)
    M, G, W = sum(sizes) + tail, len(sizes), 2 * N if gated else N
    dy, pre = torch.randn((M, N), generator=g, device=DEV), torch.randn((M, W), generator=g, device=DEV) * 3
    ends = np.cumsum(sizes)
    dy[ends[-1]:], pre[ends[-1]:] = float("nan"), float("inf")             # not read
    dy, pre = dy.to(DT[dtype]), pre.to(DT[dtype])
    offs = torch.from_numpy(ends.astype(np.int32)).to(DEV)
    dpre, dbias = mxq.mx_act_grad(dy, pre, "gelu", gated, offs)
    assert dbias.shape == (G, W) and not dpre[ends[-1]:].any()
    for e_, (r0, r1) in enumerate(ro.group_ranges(ends, M)):
        d, e = ao.grad(dy[r0:r1].double(), pre[r0:r1].double(), "gelu", gated)
        near(dpre[r0:r1], d, e, f"dpre of group {e_}")
        near(dbias[e_:e_ + 1], d.sum(0, keepdim=True), sum_error(d, e, r1 - r0, M / 16 + 1)[None], f"dbias of group {e_}")


def test_gradient_of_no_rows_and_bad_ends():
    dpre, dbias = mxq.mx_act_grad(torch.empty((0, 40), device=DEV), torch.empty((0, 80), device=DEV), "silu", True)
    assert dpre.shape == (0, 80) and not dbias.any()
    offs = torch.zeros(3, dtype=torch.int32, device=DEV)
    _, dbias = mxq.mx_act_grad(torch.empty((0, 40), device=DEV), torch.empty((0, 40), device=DEV), "silu", False, offs)
    assert dbias.shape == (3, 40) and not dbias.any()
    dy, pre = torch.randn((50, 40), device=DEV), torch.randn((50, 40), device=DEV)
    bad = [20, 7, 1000, -5]                                                 # clamped to an ascending sequence in [0, 50]
    dpre, dbias = mxq.mx_act_grad(dy, pre, "silu", False, torch.tensor(bad, dtype=torch.int32, device=DEV))
    good, gbias = mxq.mx_act_grad(dy, pre, "silu", False, torch.tensor([20, 20, 50, 50], dtype=torch.int32, device=DEV))
    assert torch.equal(dpre, good) and torch.equal(dbias, gbias)


def test_slopes_at_the_ends():
    """Infinite and large values have the slope's limits; NaN stays."""
    inf = float("inf")
    x = torch.tensor([[inf, 1e30, 200.0, 0.0, -0.0, -200.0, -1e30, -inf, float("nan")]], device=DEV)
    for act in ao.ACTS:
        d, _ = mxq.mx_act_grad(torch.ones_like(x), x, act, bias=False)
        zero = {"none": 1.0, "relu": 0.0}.get(act, 0.5)
        low = 1.0 if act == "none" else 0.0
        assert d[0, :8].tolist() == [1, 1, 1, zero, zero, low, low, low], act
        assert (d[0, 8].item() == 1) if act == "none" else d[0, 8].isnan(), act


@pytest.mark.parametrize("gated", [False, True])
def test_rows_far_apart(gated):
    """Results, residuals and kept sums 2^23 elements apart, 384 rows: offsets
    past 32 bits.  The bits are those of contiguous rows."""
    g = gen(23 + gated)
    M, N, K, far = 384, 256, 256, 1 << 23
    W = 2 * N if gated else N
    bf = torch.bfloat16
    out, res, kept, dpre = (torch.empty((M, far), dtype=bf, device=DEV)[:, 7:n + 7] for n in (N, N, W, W))
    bias = torch.randn(W, generator=g, device=DEV)
    near_res = torch.randn((M, N), generator=g, device=DEV).to(bf)
    res.copy_(near_res)
    A, B = Operand((M, K), g, K), Operand((W, K), g, K)
    qa, sa = mxq.i8_quantize_rows(torch.randn((M, K), generator=g, device=DEV))
    qb, sb = mxq.i8_quantize_rows(torch.randn((W, K), generator=g, device=DEV))
    want = mxq.i8_gemm_nt_act(qa, sa, qb, sb, bias, "gelu", gated, near_res)
    assert torch.equal(mxq.i8_gemm_nt_act(qa, sa, qb, sb, bias, "gelu", gated, res, out=out), want)
    for form in ("rows", "odd"):
        ops = (A.q, A.scales(form), B.q, B.scales(form), bias, "silu", gated)
        want, pre = mxq.mx_gemm_nt_act(*ops, near_res, pre=True)
        mxq.mx_gemm_nt_act(*ops, res, out=out, pre=kept)
        assert torch.equal(out, want) and torch.equal(kept, pre)
    want, sums = mxq.mx_act_grad(near_res, pre, "silu", gated)
    _, got = mxq.mx_act_grad(res, kept, "silu", gated, out=(dpre, None))
    assert torch.equal(dpre, want) and torch.equal(got, sums)


# ---------------------------------------------------------- streams and graphs
def test_a_training_step_in_a_graph_while_an_eager_one_is_alive():
    """Product, gradient and the products behind it, captured, replayed with new
    inputs and other work in between, and again on another stream."""
    g = gen(11)
    M, N, K = 256, 256, 512
    ops = [torch.randn((r, K), generator=g, device=DEV).bfloat16() for r in (M, 2 * N)]
    bias, dy = torch.randn(2 * N, generator=g, device=DEV), torch.randn((M, N), generator=g, device=DEV).bfloat16()

    def step(x, w, dy):
        qx, sx, _, _ = mxq.mx_quantize_2d_dual(x)
        qw, sw, _, _ = mxq.mx_quantize_2d_dual(w)
        y, pre = mxq.mx_gemm_nt_act(qx, sx, qw, sw, bias, "silu", True, pre=True)
        dpre, dbias = mxq.mx_act_grad(dy, pre, "silu", True)
        q, s = mxq.i8_quantize_rows(w)
        z = mxq.i8_linear_act(x, q, s, bias, "gelu", True, residual=y)
        return y, pre, dpre, dbias, z

    alive = step(*ops, dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*ops, dy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(*ops, dy)
    for rep in range(3):
        ops[0].copy_(torch.randn((M, K), generator=g, device=DEV))
        dy.copy_(torch.randn((M, N), generator=g, device=DEV))
        for t in held:
            t.fill_(rep)
        graph.replay()
        want = step(*ops, dy)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = step(*ops, dy)
        torch.cuda.synchronize()
        for a, b, c in zip(held, want, other):
            assert torch.equal(a, b) and torch.equal(c, b), rep
    assert all(t.isfinite().all() for t in alive)


def test_two_calls_at_once():
    """Calls whose kernels may overlap on two streams give their own results."""
    g = gen(12)
    work = []
    for M, N, K in ((300, 700, 512), (16, 4096, 2048)):
        x, b, sb = torch.randn((M, K), generator=g, device=DEV), codes((2 * N, K), g), small_scales(2 * N, K, g)
        dy, pre = torch.randn((M, N), generator=g, device=DEV), torch.randn((M, 2 * N), generator=g, device=DEV)
        work.append(lambda x=x, b=b, sb=sb, dy=dy, pre=pre: (mxq.i8_linear_act(x, b, sb, None, "silu", True),
                                                             *mxq.mx_act_grad(dy, pre, "silu", True)))
    want = [w() for w in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    got = []
    for _ in range(5):
        for s, w in zip(streams, work):
            with torch.cuda.stream(s):
                got.append(w())
    torch.cuda.synchronize()
    for i, outs in enumerate(got):
        for a, b in zip(outs, want[i % 2]):
            assert torch.equal(a, b)


def test_refusals_of_the_binding():
    g = gen(13)
    a, b, sa, sb = codes((8, 32), g), codes((6, 32), g), small_scales(8, 32, g), small_scales(6, 32, g)
    bad = [dict(act="swish"), dict(act=1), dict(bias=torch.zeros(5, device=DEV)), dict(bias=torch.zeros(6, device=DEV).double()),
           dict(bias=torch.zeros(6)), dict(gated=True, bias=torch.zeros(3, device=DEV)),
           dict(residual=torch.zeros((8, 5), device=DEV).bfloat16()), dict(residual=torch.zeros((8, 6), device=DEV)),
           dict(gated=True, residual=torch.zeros((8, 6), device=DEV).bfloat16()), dict(out_dtype=torch.float16),
           dict(out=torch.zeros((8, 5), device=DEV))]
    for kw in bad:
        with pytest.raises(ValueError):
            mxq.i8_gemm_nt_act(a, sa, b, sb, **kw)
    with pytest.raises(ValueError):
        mxq.i8_gemm_nt_act(a, sa, b[:5], sb[:5], gated=True)               # an odd number of channels
    y = torch.zeros((8, 8), device=DEV)
    with pytest.raises(mxq.MXError) as e:                                  # overlaps the result, but is not it
        mxq.i8_gemm_nt_act(a, sa, b, sb, residual=y[:, 1:7], out=y[:, :6])
    assert e.value.status == 8
    q = torch.zeros((128, 128), dtype=torch.uint8, device=DEV)
    s = torch.full((128, 4), 127, dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError):
        mxq.mx_gemm_nt_act(q, s, q, s, pre=torch.zeros((128, 128), device=DEV))    # bf16 result, fp32 pre
    with pytest.raises(mxq.MXError):
        mxq.mx_gemm_nt_act(q, s, q, s, gated=True)                         # 64 results a row
    with pytest.raises(ValueError):
        mxq.mx_act_grad(torch.zeros((4, 4), device=DEV), torch.zeros((4, 4), device=DEV), "silu", True)
    with pytest.raises(ValueError):
        mxq.mx_act_grad(torch.zeros((4, 4), device=DEV), torch.zeros((4, 4), device=DEV).bfloat16())
    x = torch.zeros((4, 4), device=DEV)
    with pytest.raises(mxq.MXError):
        mxq.mx_act_grad(torch.zeros((4, 4), device=DEV), x, out=(x, None))
