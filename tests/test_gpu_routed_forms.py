"""GPU tests of the routed-expert operators at the sizes and inputs that reach
each form of their kernels: the product's tiles, rings and splits with ragged
edges, routing over several passes and through the prefix kernel, fp32 scores
that differ in their last bits only.

Tolerances are those of the operations (test_gpu_routed derives them):
products 4 u of the magnitudes and 2^-8 |C| in bf16; weights
(6 D + 2 E + 32) u; prob adds one u for each term that may be added in turn,
64 passes within a block and its fellow blocks.
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


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def codes(shape, g):
    return torch.randint(-127, 128, shape, generator=g, device=DEV, dtype=torch.int8)


def scales(shape, g):
    return torch.exp(torch.randn(shape, generator=g, device=DEV))


def plain(a, sa, b, sb, bias=None):
    """The product in binary64 (sums of integers below 2^53: exact) and the
    magnitudes that went into it."""
    c = (a.double() @ b.double().t().contiguous()) * sa.double()[:, None] * sb.double()[None]
    mag = c.abs()
    if bias is not None:
        c, mag = c + bias.double(), mag + bias.double().abs()
    return c, mag


def near(got, want, mag, dtype, what):
    tol = 4 * U * mag + (2.0 ** -8 * want.abs() if dtype == torch.bfloat16 else 0)
    bad = ~((got.double() - want).abs() <= tol) & ~(got.isnan() & want.isnan())
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        pytest.fail(f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound; first {i}: got {got[i].item()!r} "
                    f"want {want[i].item()!r}")


def at_any_byte(t):
    """t with its base one byte past an aligned one."""
    buf = torch.empty(t.numel() + 17, dtype=t.dtype, device=DEV)
    v = buf[1:1 + t.numel()].view(t.shape)
    v.copy_(t)
    return v


# ------------------------------------------------------------------- products
# 256 CUs take one tile each of 256 x 256, 128 x 256, 128 x 128, 128 x 64 and
# 64 x 64 here; the contraction ends one piece into its last step, one before
# its end, or holds less than the stages that run ahead.
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("K", [16, 240, 1040])
@pytest.mark.parametrize("M,N", [(4000, 4040), (2000, 4040), (2001, 2040), (1000, 2039), (970, 1001), (17, 50)])
def test_dense_tiles(M, N, K, out):
    g = gen(M + N + K)
    a, b, sa, sb = codes((M, K), g), codes((N, K), g), scales(M, g), scales(N, g)
    bias = torch.randn(N, generator=g, device=DEV) * 50
    want, mag = plain(a, sa, b, sb, bias)
    buf = torch.full((M, N + 3), 99, dtype=DT[out], device=DEV)
    near(mxq.i8_gemm_nt(a, sa, b, sb, bias, out=buf[:, :N]), want, mag, DT[out], "pitched result")
    assert (buf[:, N:] == 99).all()
    near(mxq.i8_gemm_nt(a, sa, b, sb, bias, out_dtype=DT[out]), want, mag, DT[out], "whole result")


# Few rows: 16, 32 and 64 columns a workgroup by N; contractions that give some
# waves no step, and a last step of one piece.
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("K", [16, 1040, 2992])
@pytest.mark.parametrize("M", [1, 3, 16])
@pytest.mark.parametrize("N", [33, 8185, 8200, 16391, 16400])
def test_few_rows(M, N, K, out):
    g = gen(M + N + K)
    a, b, sa, sb = codes((M, K), g), codes((N, K), g), scales(M, g), scales(N, g)
    bias = torch.randn(N, generator=g, device=DEV) * 50
    want, mag = plain(a, sa, b, sb, bias)
    near(mxq.i8_gemm_nt(a, sa, b, sb, bias, out_dtype=DT[out]), want, mag, DT[out], "codes")


# Activations quantized beside the first weights (up to 16 KiB of them), or by
# a kernel of its own (beyond); rows that hold what is not finite.
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,K", [(1, 16), (1, 4096), (1, 8192), (4, 1040), (5, 816), (16, 256), (16, 512), (16, 528)])
@pytest.mark.parametrize("N", [40, 8200, 16400])
def test_few_rows_of_activations(M, K, N, dtype):
    g = gen(M + N + K)
    x = (torch.randn((M, K), generator=g, device=DEV) * scales((M, 1), g)).to(DT[dtype])
    if M > 3:
        x[1, K // 2] = float("nan")
        x[2, K - 1] = -float("inf")
        x[3] = 0
    b, sb = codes((N, K), g), scales(N, g)
    q, s = ro.quantize(x.float().cpu().numpy())
    qa, sa = torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV)
    for out in (torch.float32, torch.bfloat16):
        want, mag = plain(qa, sa, b, sb)
        got = mxq.i8_linear(x, b, sb, out_dtype=out)
        near(got, want, mag.nan_to_num(0), out, str(out))
        if M > 3:
            assert got[1:3].isnan().all() and not got[3].any()


# Few tiles: activations quantized by the product itself up to 2048 of them, at
# any element and pitch; beyond, and with more tiles, by a kernel before it.
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (17, 40, 15), (20, 300, 128), (33, 70, 129), (77, 1000, 1111), (64, 500, 1024),
                                   (5, 700, 1025), (100, 129, 2047), (40, 333, 2048), (40, 333, 2049), (300, 800, 600)])
def test_rows_of_activations(M, N, K, dtype):
    g = gen(M + N + K)
    b, sb = at_any_byte(codes((N, K), g)), scales(N, g)
    bias = torch.randn(N, generator=g, device=DEV)
    buf = torch.full((M * (K + 3) + 8,), float("nan"), dtype=DT[dtype], device=DEV)
    x = buf[1:1 + M * (K + 3)].view(M, K + 3)[:, :K]
    x.copy_(torch.randn((M, K), generator=g, device=DEV) * scales((M, 1), g))
    if M > 16:
        x[1, K - 1] = float("nan")
        x[16, K // 2] = float("inf")
        x[3] = 0
    q, s = ro.quantize(x.float().cpu().numpy())
    qa, sa = torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV)
    for bi in (None, bias):
        for out in (torch.float32, torch.bfloat16):
            want, mag = plain(qa, sa, b, sb, bi)
            near(mxq.i8_linear(x, b, sb, bi, out_dtype=out), want, mag.nan_to_num(0), out, str(out))


# Rows that start at any byte: waves that split the contraction in 16 x 16 and
# 64 x 32, and 128 x 128 tiles.
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 3000, 1041), (70, 900, 257), (300, 1500, 1041), (511, 2100, 333), (2000, 2100, 517), (130, 1300, 7)])
def test_rows_at_any_byte(M, N, K, out):
    g = gen(M + N + K)
    a, b = at_any_byte(codes((M, K), g)), at_any_byte(codes((N, K), g))
    sa, sb = scales(M, g), scales(N, g)
    want, mag = plain(a, sa, b, sb)
    near(mxq.i8_gemm_nt(a, sa, b, sb, out_dtype=DT[out]), want, mag, DT[out], "any byte")


# Mean rows of a group up to 16, 160 and beyond (whole pieces), up to 18 and
# beyond (any byte); empty groups, single rows, a tail.
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("N,K", [(300, 272), (513, 1040), (40, 16)])
@pytest.mark.parametrize("sizes,tail", [
    ([0, 3, 16, 1, 0, 40, 17, 15], 4), ([0, 0, 0, 1], 0), ([100, 0, 257, 128, 1, 65], 60), ([700, 0, 3, 513, 256], 100),
    ([5] * 100, 0), ([0, 1000], 0)])
def test_groups(sizes, tail, N, K, out):
    g = gen(sum(sizes) + N)
    M, G = sum(sizes) + tail, len(sizes)
    a, b, sa, sb = codes((M, K), g), codes((G, N, K), g), scales(M, g), scales((G, N), g)
    offs = np.cumsum(sizes)
    want, mag = torch.zeros((M, N), dtype=torch.float64, device=DEV), torch.zeros((M, N), dtype=torch.float64, device=DEV)
    for e, (r0, r1) in enumerate(ro.group_ranges(offs, M)):
        want[r0:r1], mag[r0:r1] = plain(a[r0:r1], sa[r0:r1], b[e], sb[e])
    sa[offs[-1]:] = float("inf")                     # the tail is no group's
    od = torch.from_numpy(offs.astype(np.int32)).to(DEV)
    near(mxq.i8_grouped_gemm_rows(a, sa, b, sb, od, out_dtype=DT[out]), want, mag, DT[out], "whole pieces")
    near(mxq.i8_grouped_gemm_rows(at_any_byte(a), sa, at_any_byte(b), sb, od, out_dtype=DT[out]), want, mag, DT[out], "any byte")


# Rows so far apart that a tile's offsets leave 32 bits.
@pytest.mark.parametrize("K", [64, 1041])
@pytest.mark.parametrize("wide", ["A", "B"])
def test_rows_far_apart(wide, K):
    M, N, pitch = (130, 70, 2 ** 24 + 16) if wide == "A" else (70, 130, 2 ** 24 + 16)
    g = gen(K)
    a, b, sa, sb = codes((M, K), g), codes((N, K), g), scales(M, g), scales(N, g)
    buf = torch.empty(130 * pitch, dtype=torch.int8, device=DEV)
    v = buf.as_strided((130, K), (pitch, 1))
    v.copy_(a if wide == "A" else b)
    A, B = (v, b) if wide == "A" else (a, v)
    want, mag = plain(a, sa, b, sb)
    near(mxq.i8_gemm_nt(A, sa, B, sb), want, mag, torch.bfloat16, "dense")
    ends = [0, 33, 34, M - 5]
    offs = torch.tensor(ends, dtype=torch.int32, device=DEV)
    want, mag = plain(a, sa, b, sb)
    want[M - 5:] = mag[M - 5:] = 0
    got = mxq.i8_grouped_gemm_rows(A, sa, B.as_strided((4, N, K), (0, B.stride(0), 1)), sb.expand(4, N), offs)
    near(got, want, mag, torch.bfloat16, "by expert")


# -------------------------------------------------------------------- routing
def plain_route(z, k, normalize, align, M):
    """Routing by sorts and sums in binary64 on the device (no invalid token,
    no bad score)."""
    T, E = z.shape
    z = z.double()
    top, order = torch.sort(z, dim=1, descending=True, stable=True)       # equal scores: lowest expert first
    taken = top[:, :k] > -torch.inf
    idx = torch.where(taken, order[:, :k], -1)
    live = z.max(1).values > -torch.inf
    p = torch.exp(z - z.max(1, keepdim=True).values).masked_fill(~live[:, None], 0)
    w = p.gather(1, order[:, :k]) * taken
    den = w.sum(1, keepdim=True) if normalize else p.sum(1, keepdim=True)
    w = (w / den).masked_fill(~live[:, None], 0)
    p = (p / p.sum(1, keepdim=True)).masked_fill(~live[:, None], 0)
    n = max(int(live.sum()), 1)
    counts = torch.stack([(idx == e).sum() for e in range(E)])
    ends = (-(-counts // align) * align).cumsum(0)
    slot = torch.full_like(idx, -1)
    src = torch.full((M,), -1, dtype=torch.int64, device=z.device)
    begin = 0
    for e in range(E):                                                     # in token order
        at = (idx.reshape(-1) == e).nonzero()[:, 0]
        to = begin + torch.arange(len(at), device=z.device)
        slot.view(-1)[at] = to
        src[to] = at
        begin = int(ends[e])
    prob = p.sum(0) / n
    loss = E * (counts / (k * n) * prob).sum()
    return dict(idx=idx, weight=w, slot=slot, src=src, counts=counts, offs=ends, live=n if live.any() else 0, prob=prob,
                loss=loss)


def check_route(z, k, normalize, align, terms):
    T, E = z.shape
    r = mxq.mx_route(z, k, normalize=normalize, align=align)
    w = plain_route(z, k, normalize, align, r.rows)
    for n in ("idx", "slot", "src", "counts", "offs"):
        assert torch.equal(getattr(r, n).long(), w[n].long()), n
    assert int(r.live) == w["live"]
    fin = torch.where(z > -torch.inf, z.double(), torch.inf)
    d = z.double().max(1).values - fin.min(1).values
    e = (6 * float(d[d > -torch.inf].max()) + 2 * E + 32) * U
    assert ((r.weight - w["weight"]).abs() <= w["weight"] * e + 2.0 ** -120).all()
    assert ((r.prob - w["prob"]).abs() <= w["prob"] * (e + terms * U) + 2.0 ** -120).all()
    assert abs(float(r.loss) - float(w["loss"])) <= float(w["loss"]) * (e + (terms + E) * U) + 2.0 ** -120


# One to four tokens, one block, its neighbours, blocks of one pass and of two,
# counts that every block adds itself and that a kernel adds for all, and the
# most passes (past 2^24 tokens).
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,k,align", [
    (1, 7, 3, 1), (4, 256, 8, 16), (5, 256, 8, 16), (64, 1024, 16, 1), (65, 1024, 16, 4), (2048, 1000, 3, 1),
    (2049, 1024, 2, 128), (8192, 256, 8, 128), (8193, 256, 8, 1), (32768, 16, 4, 1), (32769, 5, 2, 128),
    (40001, 300, 4, 8), (262200, 16, 1, 1), (2 ** 24 + 4097, 3, 2, 128)])
def test_route_by_size(T, E, k, align, dtype):
    g = gen(T + E)
    z = (torch.randn((T, E), generator=g, device=DEV) * 2).to(DT[dtype])
    z.masked_fill_(torch.rand((T, E), generator=g, device=DEV) < 0.05, -torch.inf)
    passes = 1 if T <= 32768 else 2 if T <= 2 ** 24 else 64
    check_route(z, k, True, align, 64 * passes + -(-T // (64 * passes)))


# fp32 scores whose first 22 bits agree: everywhere in a row, at the last pick
# and its successor only, or between picks only; rows of each kind meet in a
# wave, which takes four.
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("E,k", [(5, 2), (16, 16), (60, 8), (64, 1), (256, 8), (300, 9), (1024, 16)])
@pytest.mark.parametrize("T", [3, 70, 3000])
def test_scores_that_differ_in_their_last_bits(T, E, k, sign):
    g = np.random.default_rng(T + E)
    order = np.argsort(g.random((T, E)), 1).astype(np.float64)            # a permutation of each row
    far = sign * (1 + order * 2.0 ** -5)                                  # apart in 22 bits, up to 33
    fine = sign * (1 + order * 2.0 ** -23)                                # E ulps of one another
    kind = np.arange(T) % 5 if T > 3 else np.array([1, 2, 3])
    rank = np.argsort(np.argsort(-far, 1), 1)
    z = far.copy()
    z[kind == 1] = fine[kind == 1]
    last, nxt = (np.where(rank == r)[1] if r < E else None for r in (k - 1, k))
    for t in range(T):
        if kind[t] == 2 and k < E:                                        # the successor one ulp below the last pick
            z[t, nxt[t]] = np.nextafter(np.float32(z[t, last[t]]), np.float32(-100))
        if kind[t] == 3:                                                  # the best two one ulp apart, the second first
            a, b = np.where(rank[t] == 0)[0][0], np.where(rank[t] == 1)[0][0]
            z[t, b] = np.nextafter(np.float32(z[t, a]), np.float32(100))
        if kind[t] == 4:                                                  # equal in all bits
            z[t] = z[t, 0]
    zd = torch.from_numpy(z.astype(np.float32)).to(DEV)
    check_route(zd, k, True, 4, 64 + -(-T // 64))
    check_route(zd, k, False, 1, 64 + -(-T // 64))


# The best k + 1 scores of a row in one lane's experts, the last two of them
# equal in their first 22 bits and out of the experts' order: a lane that keeps k
# keys has dropped the one that shows it.
@pytest.mark.parametrize("E,k,lane", [(256, 8, [0, 1, 2, 3, 64, 65, 66, 67, 128]), (512, 8, [4, 5, 6, 7, 68, 69, 70, 71, 132]),
                                      (1024, 16, [b + i for b in (8, 72, 136, 200) for i in range(4)] + [264]),
                                      (512, 16, [b + i for b in (8, 72, 136, 200) for i in range(4)] + [264]),
                                      (1000, 8, [60, 61, 62, 63, 124, 125, 126, 127, 188])])
def test_best_scores_in_one_lane(E, k, lane):
    assert len(lane) == k + 1
    z = np.full((70, E), -4.0, np.float32) - np.arange(E, dtype=np.float32) * 2.0 ** -10
    g = np.random.default_rng(E)
    for t in range(70):
        order = g.permutation(k + 1)
        low, high = min(order[-2:]), max(order[-2:])
        for i, j in enumerate(order[:-2]):
            z[t, lane[j]] = 8 - i * 0.25
        z[t, lane[high]] = np.nextafter(np.float32(1), np.float32(2))      # the last pick: the later expert
        z[t, lane[low]] = 1
    check_route(torch.from_numpy(z).to(DEV), k, True, 1, 64 + 2)


# More tokens than the gradient's grid takes at once (4096 workgroups of 16).
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradient_of_many_tokens(dtype, normalize):
    T, E, k = 70001, 12, 3
    g = gen(5)
    z = (torch.randn((T, E), generator=g, device=DEV) * 2).to(DT[dtype])
    r = mxq.mx_route(z, k, normalize=normalize)
    w = plain_route(z, k, normalize, 1, r.rows)
    up = torch.randn((T, k), generator=g, device=DEV)
    got = mxq.mx_route_grad(z, r, up, torch.full((1,), 0.37, device=DEV)).double()
    p = torch.softmax(z.double(), 1)
    a = 0.37 * E * w["counts"].double() / (k * T) / T
    a = a.expand(T, E).clone()
    u = torch.zeros((T, E), dtype=torch.float64, device=DEV).scatter_(1, w["idx"], up.double())
    v = torch.zeros((T, E), dtype=torch.float64, device=DEV).scatter_(1, w["idx"], w["weight"])
    want, mag = torch.zeros_like(p), torch.zeros_like(p)
    if normalize:
        want = v * (u - (v * u).sum(1, keepdim=True))
        mag = v * (u.abs() + (v * u.abs()).sum(1, keepdim=True))
    else:
        a += u
    want += p * (a - (p * a).sum(1, keepdim=True))
    mag += p * (a.abs() + (p * a.abs()).sum(1, keepdim=True))
    D = float((z.double().max(1).values - z.double().min(1).values).max())
    tol = mag * (12 * D + 6 * E + 64) * U + 2.0 ** -120 + (2.0 ** -8 * want.abs() if dtype == "bf16" else 0)
    assert ((got - want).abs() <= tol).all()
