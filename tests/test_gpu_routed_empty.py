"""GPU tests of the routed-expert operators where a batch has no tokens but the
padded buffer has rows (rows without a token are 0 all the same), or where rows
have no elements (what does not depend on them is written all the same)."""
import pytest
import torch

import mx9_dual_axis_amd as mxq
from helpers import require_gpu, say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _gpu(request):
    require_gpu()
    say(request.node.name)


def empty_map(M, k=3):
    """The map of no tokens to M rows."""
    return (torch.empty((0, k), dtype=torch.int32, device=DEV), torch.full((M,), -1, dtype=torch.int32, device=DEV))


# A row of codes of 0 has the scale of the smallest magnitude that quantization
# takes, 127 2^-126 / 127, whatever the row's length.
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [1, 15, 40, 5000])
@pytest.mark.parametrize("M", [1, 5, 16, 33])
def test_quantized_rows_of_no_tokens(M, K, dtype):
    slot, src = empty_map(M)
    x = torch.empty((0, K), dtype=DT[dtype], device=DEV)
    q = torch.full((M, K + 3), 99, dtype=torch.int8, device=DEV)
    s = torch.full((M,), float("nan"), device=DEV)
    mxq.mx_dispatch_i8(x, slot, src, out=(q[:, :K], s))
    assert not q[:, :K].any() and (q[:, K:] == 99).all()
    assert (s == 2.0 ** -126).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [1, 40, 5000])
@pytest.mark.parametrize("M", [1, 5, 33])
def test_rows_and_gradient_rows_of_no_tokens(M, N, dtype):
    slot, src = empty_map(M)
    none = torch.empty((0, N), dtype=DT[dtype], device=DEV)
    out = torch.full((M, N + 3), 99, dtype=DT[dtype], device=DEV)
    mxq.mx_dispatch(none, slot, src, out=out[:, :N])
    assert not out[:, :N].any() and (out[:, N:] == 99).all()
    out.fill_(99)
    rows = torch.ones((M, N), dtype=DT[dtype], device=DEV)
    drows, dweight = mxq.mx_combine_grad(none, rows, slot, None, src, out=(out[:, :N], None))
    assert not drows.any() and (out[:, N:] == 99).all() and dweight.shape == (0, 3)
    assert mxq.mx_combine(rows, slot).shape == (0, N)


# A row of no elements has the scale of the smallest magnitude, like a row of
# zeros; the inner product of two of them is 0.
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,M", [(0, 5), (1, 1), (7, 20), (40, 130)])
def test_rows_of_no_elements(T, M, dtype):
    k = 2
    slot = torch.arange(T * k, dtype=torch.int32, device=DEV).reshape(T, k)
    slot[slot >= M] = -1
    src = torch.arange(M, dtype=torch.int32, device=DEV)
    src[src >= T * k] = -1
    x = torch.empty((T, 0), dtype=DT[dtype], device=DEV)
    for call, n in ((lambda o: mxq.mx_dispatch_i8(x, slot, src, out=o), M), (lambda o: mxq.i8_quantize_rows(x, out=o), T)):
        s = torch.full((n,), float("nan"), device=DEV)
        q, _ = call((torch.empty((n, 0), dtype=torch.int8, device=DEV), s))
        assert q.shape == (n, 0) and (s == 2.0 ** -126).all()
    rows = torch.empty((M, 0), dtype=DT[dtype], device=DEV)
    weight, dweight = torch.ones((T, k), device=DEV), torch.full((T, k), float("nan"), device=DEV)
    drows, _ = mxq.mx_combine_grad(x, rows, slot, weight, src, out=(None, dweight))
    assert drows.shape == (M, 0) and not dweight.any()
    assert mxq.mx_dispatch(x, slot, src).shape == (M, 0) and mxq.mx_combine(rows, slot, weight).shape == (T, 0)


# ... and the product of no codes is the bias.
@pytest.mark.parametrize("M,N", [(1, 40), (17, 33), (300, 700)])
def test_products_of_no_codes(M, N):
    B, sB, bias = torch.empty((N, 0), dtype=torch.int8, device=DEV), torch.ones(N, device=DEV), torch.randn(N, device=DEV)
    A, x = torch.empty((M, 0), dtype=torch.int8, device=DEV), torch.empty((M, 0), device=DEV)
    want = bias.expand(M, N)
    assert torch.equal(mxq.i8_gemm_nt(A, torch.ones(M, device=DEV), B, sB, bias, out_dtype=torch.float32), want)
    assert torch.equal(mxq.i8_linear(x, B, sB, bias), want)
    assert not mxq.i8_linear(x, B, sB).any()
