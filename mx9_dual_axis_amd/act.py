"""Binding of ``include/mxq_act.h``: products with bias, activation and residual
in their epilogue, and its gradient.

  i8_linear_act(x, B, sB, ...)                      -> y, i8_linear with the epilogue
  i8_gemm_nt_act(A, sA, B, sB, ...)                 -> y, i8_gemm_nt
  i8_grouped_gemm_rows_act(A, sA, B, sB, offs, ...) -> y, i8_grouped_gemm_rows
  mx_gemm_nt_act(A, sA, B, sB, ...)                 -> y or (y, pre), mx_gemm_nt
  mx_grouped_gemm_rows_act(A, sA, B, sB, offs, ...) -> y or (y, pre), mx_grouped_gemm_rows
  mx_gemm_nt_act_mfma, mx_grouped_gemm_rows_act_mfma   (scales in the matrix-core layout)
  mx_act_grad(dy, pre, act, gated, offs)            -> (dpre, dbias)

x = sum + bias; y = act(x) (+ residual), or with gated=True, where B holds the
gates' channels and then as many more, y = act(x[:, :N]) * x[:, N:] (+
residual).  act is "none", "relu", "silu", "gelu" or "gelu_tanh".  bias is
float32 (a row for each expert in the grouped calls), residual has the
result's shape and dtype and may be `out` itself.

The 8-bit sums are exact, so a row's bits depend on that row alone.  The MXFP8
sums are added in an order that depends on the call's sizes: the same call gives
the same bits, but a row's may differ between batch sizes, and from those of
mx_gemm_nt and mx_grouped_gemm_rows.
"""
from __future__ import annotations

import ctypes

import torch

from .routed import _ESZ, _F32, _I8, _flat, _matrix, _out_matrix, _run
from .routed import _product_out

ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}

_lib = None


def _L():
    global _lib
    if _lib is None:
        from . import library

        lib = library()
        P, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
        lib.i8_gemm_nt_act.argtypes = [P, I64, P, P, I64, P, I64, I64, I64, I32, I32, P, P, I64, P, I64, I32, P]
        lib.i8_linear_act.argtypes = [P, I32, I64, P, I64, P, I64, I64, I64, I32, I32, P, P, I64, P, I64, I32, P, I64, P]
        lib.i8_grouped_gemm_rows_act.argtypes = [P, I64, P, P, I64, I64, P, I64, P, I32, I64, I64, I64, I32, I32, P, I64,
                                                 P, I64, I32, P]
        lib.mx_gemm_nt_act.argtypes = [P, I64, P, I64, I64, P, I64, P, I64, I64, I64, I64, I64, I32, I32, P, P, I64, P,
                                       I64, P, I64, I32, P]
        lib.mx_gemm_nt_act_mfma.argtypes = [P, I64, P, P, I64, P, I64, I64, I64, I32, I32, P, P, I64, P, I64, P, I64, I32,
                                            P]
        lib.mx_grouped_gemm_rows_act.argtypes = [P, I64, P, I64, I64, P, I64, I64, P, I64, I64, I64, P, I32, I64, I64,
                                                 I64, I32, I32, P, I64, P, I64, P, I64, I32, P]
        lib.mx_grouped_gemm_rows_act_mfma.argtypes = [P, I64, P, P, I64, I64, P, I64, P, I32, I64, I64, I64, I32, I32, P,
                                                      I64, P, I64, P, I64, I32, P]
        lib.mx_act_grad_workspace.argtypes = [I64, I64, I32, I32, I32]
        lib.mx_act_grad_workspace.restype = I64
        lib.mx_act_grad.argtypes = [P, I64, P, I64, I32, I64, I64, I32, I32, P, I32, P, I64, P, P, I64, P]
        for f in (lib.i8_gemm_nt_act, lib.i8_linear_act, lib.i8_grouped_gemm_rows_act, lib.mx_gemm_nt_act,
                  lib.mx_gemm_nt_act_mfma, lib.mx_grouped_gemm_rows_act, lib.mx_grouped_gemm_rows_act_mfma,
                  lib.mx_act_grad):
            f.restype = ctypes.c_int
        _lib = lib
    return _lib


def _act(act):
    code = ACTS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {', '.join(ACTS)}, not {act!r}")
    return code


def _results(W, gated):
    if not gated:
        return W
    if W % 2:
        raise ValueError(f"a gated product needs an even number of B's channels, not {W}")
    return W // 2


def _bias(bias, W, i):
    return None if bias is None else _flat(bias, "bias", _F32, (W,), i)


def _expert_bias(bias, G, W, i):
    """(pointer, elements from one expert's to the next)"""
    if bias is None:
        return None, 0
    if not isinstance(bias, torch.Tensor) or bias.dtype is not _F32 or bias.dim() != 2 or bias.shape[0] < G or (
            bias.shape[1] != W) or bias.get_device() != i or (W > 1 and bias.stride(1) != 1):
        raise ValueError(f"bias must be a float32 [E >= {G}, {W}] tensor with contiguous rows on the device of A")
    return bias.data_ptr(), bias.stride(0)


def _residual(residual, shape, dtype, i):
    """(pointer, row pitch)"""
    if residual is None:
        return None, 0
    pitch = _matrix(residual, "residual", (dtype,), i)[0]
    if residual.shape != shape:
        raise ValueError(f"residual must have shape {tuple(shape)}, not {tuple(residual.shape)}")
    return residual.data_ptr(), pitch


def i8_gemm_nt_act(A: torch.Tensor, sA: torch.Tensor, B: torch.Tensor, sB: torch.Tensor, bias: torch.Tensor | None = None,
                   act: str = "none", gated: bool = False, residual: torch.Tensor | None = None,
                   out_dtype=torch.bfloat16, out: torch.Tensor | None = None):
    """i8_gemm_nt with the epilogue: A [M, K], B [W, K] int8 codes, y [M, N]."""
    lda, M, K = _matrix(A, "A", (_I8,))
    i = A.get_device()
    ldb, W, KB = _matrix(B, "B", (_I8,), i)
    if KB != K:
        raise ValueError("A and B must share the contraction extent")
    code, N = _act(act), _results(W, gated)
    sa, sb, bi = _flat(sA, "sA", _F32, (M,), i), _flat(sB, "sB", _F32, (W,), i), _bias(bias, W, i)
    out, ldc = _product_out(out, (M, N), out_dtype, A)
    res, ld_r = _residual(residual, (M, N), out.dtype, i)
    _run(i, _L().i8_gemm_nt_act, A.data_ptr(), lda, sa, B.data_ptr(), ldb, sb, M, N, K, code, 1 if gated else 0, bi, res,
         ld_r, out.data_ptr(), ldc, _ESZ[out.dtype])
    return out


def i8_linear_act(x: torch.Tensor, B: torch.Tensor, sB: torch.Tensor, bias: torch.Tensor | None = None, act: str = "none",
                  gated: bool = False, residual: torch.Tensor | None = None, out_dtype=None,
                  out: torch.Tensor | None = None):
    """i8_linear with the epilogue: x [M, K] float32 or bfloat16, quantized by
    rows on the way; the result has x's dtype unless out_dtype or out says
    otherwise."""
    ld, M, K = _matrix(x, "x", _ESZ)
    i = x.get_device()
    ldb, W, KB = _matrix(B, "B", (_I8,), i)
    if KB != K:
        raise ValueError("x and B must share the contraction extent")
    code, N = _act(act), _results(W, gated)
    sb, bi = _flat(sB, "sB", _F32, (W,), i), _bias(bias, W, i)
    out, ldc = _product_out(out, (M, N), out_dtype or x.dtype, x)
    res, ld_r = _residual(residual, (M, N), out.dtype, i)
    size = M * ((K + 15) // 16 * 16) + (M * 4 + 15) // 16 * 16
    ws = x.new_empty_strided((size,), (1,), dtype=torch.uint8)
    _run(i, _L().i8_linear_act, x.data_ptr(), _ESZ[x.dtype], ld, B.data_ptr(), ldb, sb, M, N, K, code, 1 if gated else 0,
         bi, res, ld_r, out.data_ptr(), ldc, _ESZ[out.dtype], ws.data_ptr(), size)
    return out


def _offs(offs, E, i):
    """(pointer, G)"""
    if not isinstance(offs, torch.Tensor) or offs.dim() != 1 or not 1 <= offs.shape[0] <= E:
        raise ValueError("offs must be an int32 [G] tensor with 1 <= G <= E")
    G = offs.shape[0]
    return _flat(offs, "offs", torch.int32, (G,), i), G


def i8_grouped_gemm_rows_act(A: torch.Tensor, sA: torch.Tensor, B: torch.Tensor, sB: torch.Tensor, offs: torch.Tensor,
                             bias: torch.Tensor | None = None, act: str = "none", gated: bool = False,
                             out_dtype=torch.bfloat16, out: torch.Tensor | None = None):
    """i8_grouped_gemm_rows with the epilogue: B [E, W, K], sB [E, W], bias
    [E, W]; rows from offs[-1] on give 0."""
    lda, M, K = _matrix(A, "A", (_I8,))
    i = A.get_device()
    if not isinstance(B, torch.Tensor) or B.dtype is not _I8 or B.dim() != 3 or B.get_device() != i:
        raise ValueError("B must be int8 [E, W, K] codes on the device of A")
    E, W, KB = B.shape
    b_gs, ldb, step = B.stride()
    if KB != K or (K > 1 and step != 1) or (W > 1 and ldb < K):
        raise ValueError("B must be [E, W, K] codes with contiguous rows that share A's contraction extent")
    if not isinstance(sB, torch.Tensor) or sB.dtype is not _F32 or sB.shape != (E, W) or sB.get_device() != i or (
            W > 1 and sB.stride(1) != 1):
        raise ValueError("sB must be a float32 [E, W] tensor with contiguous rows")
    code, N = _act(act), _results(W, gated)
    of, G = _offs(offs, E, i)
    sa = _flat(sA, "sA", _F32, (M,), i)
    bi, bi_gs = _expert_bias(bias, G, W, i)
    out, ldc = _product_out(out, (M, N), out_dtype, A)
    _run(i, _L().i8_grouped_gemm_rows_act, A.data_ptr(), lda, sa, B.data_ptr(), ldb if ldb > K else K, b_gs, sB.data_ptr(),
         sB.stride(0), of, G, M, N, K, code, 1 if gated else 0, bi, bi_gs, out.data_ptr(), ldc, _ESZ[out.dtype])
    return out


# ---- MXFP8 ----
_E4M3 = (torch.uint8, torch.float8_e4m3fn)


def _scales(s, shape, name, i):
    if not isinstance(s, torch.Tensor) or s.dtype is not torch.uint8 or s.shape != shape or s.get_device() != i:
        raise ValueError(f"{name} must be a uint8 {list(shape)} view on the device of A")
    return s.stride()


def _mfma_scales(s, n, name, i):
    if not isinstance(s, torch.Tensor) or s.dtype is not torch.uint8 or not s.is_contiguous() or s.numel() != n or (
            s.get_device() != i):
        raise ValueError(f"{name} must be {n} contiguous uint8 scales in the matrix-core layout on the device of A")


def _kept(pre, shape, dtype, like):
    """(pre or None, pointer, pitch)"""
    if pre is None or pre is False:
        return None, None, 0
    pre, pitch = _out_matrix(None if pre is True else pre, "pre", shape, dtype, like)
    return pre, pre.data_ptr(), pitch


def _mx_dense(A, sA, B, sB, bias, act, gated, residual, out_dtype, out, pre, mfma):
    lda, M, K = _matrix(A, "A", _E4M3)
    i = A.get_device()
    ldb, W, KB = _matrix(B, "B", _E4M3, i)
    if KB != K:
        raise ValueError("A and B must share the contraction extent")
    code, N = _act(act), _results(W, gated)
    bi = _bias(bias, W, i)
    out, ldc = _product_out(out, (M, N), out_dtype, A)
    res, ld_r = _residual(residual, (M, N), out.dtype, i)
    pre, pp, ld_p = _kept(pre, (M, W), out.dtype, A)
    rest = (M, N, K, code, 1 if gated else 0, bi, res, ld_r, out.data_ptr(), ldc, pp, ld_p, _ESZ[out.dtype])
    if mfma:
        _mfma_scales(sA, M * (K // 32), "sA", i)
        _mfma_scales(sB, W * (K // 32), "sB", i)
        _run(i, _L().mx_gemm_nt_act_mfma, A.data_ptr(), lda, sA.data_ptr(), B.data_ptr(), ldb, sB.data_ptr(), *rest)
    else:
        sa, sb = _scales(sA, (M, K // 32), "sA", i), _scales(sB, (W, K // 32), "sB", i)
        _run(i, _L().mx_gemm_nt_act, A.data_ptr(), lda, sA.data_ptr(), *sa, B.data_ptr(), ldb, sB.data_ptr(), *sb, *rest)
    return out if pre is None else (out, pre)


def mx_gemm_nt_act(A: torch.Tensor, sA: torch.Tensor, B: torch.Tensor, sB: torch.Tensor, bias: torch.Tensor | None = None,
                   act: str = "none", gated: bool = False, residual: torch.Tensor | None = None,
                   out_dtype=torch.bfloat16, out: torch.Tensor | None = None, pre=None):
    """mx_gemm_nt with the epilogue: A [M, K], B [W, K] E4M3 codes with scale
    views sA [M, K/32], sB [W, K/32].  pre=True, or a tensor [M, W] of the
    result's dtype, keeps x for mx_act_grad: (y, pre) is returned then."""
    return _mx_dense(A, sA, B, sB, bias, act, gated, residual, out_dtype, out, pre, False)


def mx_gemm_nt_act_mfma(A: torch.Tensor, sA: torch.Tensor, B: torch.Tensor, sB: torch.Tensor,
                        bias: torch.Tensor | None = None, act: str = "none", gated: bool = False,
                        residual: torch.Tensor | None = None, out_dtype=torch.bfloat16, out: torch.Tensor | None = None,
                        pre=None):
    """mx_gemm_nt_act with both scales in the matrix-core layout."""
    return _mx_dense(A, sA, B, sB, bias, act, gated, residual, out_dtype, out, pre, True)


def _mx_grouped(A, sA, B, sB, offs, bias, act, gated, out_dtype, out, pre, mfma):
    lda, M, K = _matrix(A, "A", _E4M3)
    i = A.get_device()
    if not isinstance(B, torch.Tensor) or B.dtype not in _E4M3 or B.dim() != 3 or B.get_device() != i:
        raise ValueError("B must be [E, W, K] E4M3 codes on the device of A")
    E, W, KB = B.shape
    b_gs, ldb, step = B.stride()
    if KB != K or (K > 1 and step != 1):
        raise ValueError("B must be [E, W, K] codes with contiguous rows that share A's contraction extent")
    code, N = _act(act), _results(W, gated)
    of, G = _offs(offs, E, i)
    bi, bi_gs = _expert_bias(bias, G, W, i)
    out, ldc = _product_out(out, (M, N), out_dtype, A)
    pre, pp, ld_p = _kept(pre, (M, W), out.dtype, A)
    rest = (of, G, M, N, K, code, 1 if gated else 0, bi, bi_gs, out.data_ptr(), ldc, pp, ld_p, _ESZ[out.dtype])
    if mfma:
        each = W * (K // 32)
        _mfma_scales(sA, M * (K // 32), "sA", i)
        _mfma_scales(sB, E * each, "sB", i)
        _run(i, _L().mx_grouped_gemm_rows_act_mfma, A.data_ptr(), lda, sA.data_ptr(), B.data_ptr(), ldb, b_gs,
             sB.data_ptr(), each, *rest)
    else:
        sa, sb = _scales(sA, (M, K // 32), "sA", i), _scales(sB, (E, W, K // 32), "sB", i)
        _run(i, _L().mx_grouped_gemm_rows_act, A.data_ptr(), lda, sA.data_ptr(), *sa, B.data_ptr(), ldb, b_gs,
             sB.data_ptr(), sb[1], sb[2], sb[0], *rest)
    return out if pre is None else (out, pre)


def mx_grouped_gemm_rows_act(A: torch.Tensor, sA: torch.Tensor, B: torch.Tensor, sB: torch.Tensor, offs: torch.Tensor,
                             bias: torch.Tensor | None = None, act: str = "none", gated: bool = False,
                             out_dtype=torch.bfloat16, out: torch.Tensor | None = None, pre=None):
    """mx_grouped_gemm_rows with the epilogue: B [E, W, K] codes, sB [E, W,
    K/32] view, bias [E, W]; rows from offs[-1] on give 0, in pre too."""
    return _mx_grouped(A, sA, B, sB, offs, bias, act, gated, out_dtype, out, pre, False)


def mx_grouped_gemm_rows_act_mfma(A: torch.Tensor, sA: torch.Tensor, B: torch.Tensor, sB: torch.Tensor,
                                  offs: torch.Tensor, bias: torch.Tensor | None = None, act: str = "none",
                                  gated: bool = False, out_dtype=torch.bfloat16, out: torch.Tensor | None = None,
                                  pre=None):
    """mx_grouped_gemm_rows_act with both scales in the matrix-core layout."""
    return _mx_grouped(A, sA, B, sB, offs, bias, act, gated, out_dtype, out, pre, True)


def mx_act_grad(dy: torch.Tensor, pre: torch.Tensor, act: str = "none", gated: bool = False,
                offs: torch.Tensor | None = None, bias: bool = True, out=None):
    """(dpre, dbias) of an epilogue for dy [M, N] and the kept pre [M, W] of one
    dtype: dpre [M, W] in that dtype; dbias float32 [W], or [G, W] by the rows
    of each group with offs, the sums of dpre before it is rounded; None when
    not `bias`.  Rows from offs[-1] on give 0."""
    ld_y, M, N = _matrix(dy, "dy", _ESZ)
    i = dy.get_device()
    ld_p, rows, W = _matrix(pre, "pre", (dy.dtype,), i)
    code = _act(act)
    if rows != M or W != (2 * N if gated else N):
        raise ValueError(f"pre must be [{M}, {2 * N if gated else N}], not {tuple(pre.shape)}")
    of, G = (None, 0) if offs is None else _offs(offs, 65535, i)
    dpre, dbias = out if out is not None else (None, None)
    dpre, ld_d = _out_matrix(dpre, "out[0]", (M, W), dy.dtype, dy)
    db, ws, size = None, None, 0
    if bias:
        shape = (W,) if offs is None else (G, W)
        if dbias is None:
            dbias = dy.new_empty_strided(shape, (1,) if offs is None else (W, 1), dtype=_F32)
        db = _flat(dbias, "out[1]", _F32, shape, i)
        size = _L().mx_act_grad_workspace(M, N, _ESZ[dy.dtype], 1 if gated else 0, G)
        if size < 0:
            raise ValueError(f"no gradient of M={M}, N={N}, G={G}")
        ws = dy.new_empty_strided((size,), (1,), dtype=torch.uint8)
    elif dbias is not None:
        raise ValueError("out[1] is for the bias's gradient, which is not asked for")
    _run(i, _L().mx_act_grad, dy.data_ptr(), ld_y, pre.data_ptr(), ld_p, _ESZ[dy.dtype], M, N, code, 1 if gated else 0, of,
         G, dpre.data_ptr(), ld_d, db, None if ws is None else ws.data_ptr(), size)
    return dpre, dbias if bias else None
