"""Binding of ``include/mxq_routed.h`` and ``include/mxq_scored.h``: routing,
dispatch, 8-bit integer products and combine of a routed-expert layer.

  mx_routing(T, E, k, align)              -> an MXRouting, the outputs and workspace of mx_route
  mx_route(logits, k, valid)              -> MXRouting (idx, weight, slot, src, counts, offs, live, prob, loss)
  mx_route_grad(logits, routing, dweight, dloss, valid) -> dlogits
  mx_route_scored(logits, k, bias, ...)   -> MXRouting, by sigmoid or softmax scores with a bias and groups
  mx_route_scored_grad(logits, routing, dweight, dloss, valid) -> dlogits
  mx_route_bias_step(bias, counts, rate)  -> the next bias
  mx_dispatch(x, slot, src)               -> rows of the padded buffer
  mx_dispatch_i8(x, slot, src)            -> (q, s), the same rows as int8 codes and scales
  i8_quantize_rows(x)                     -> (q, s)
  i8_gemm_nt(A, sA, B, sB, bias)          -> C = A B^T
  i8_linear(x, B, sB, bias)               -> the product of x, quantized on the way
  i8_grouped_gemm_rows(A, sA, B, sB, offs) -> C, each group's rows with its expert's B[g]
  mx_combine(rows, slot, weight)          -> y, the weighted sum of each token's expert rows
  mx_combine_grad(dy, rows, slot, weight, src) -> (drows, dweight)

As in the package's other calls, every step runs in the library's kernels on
the current stream, outputs are allocated with torch unless `out` is given,
and a refused call raises before anything is launched.
"""
from __future__ import annotations

import torch

_ESZ = {torch.float32: 0, torch.bfloat16: 1}      # MX_DTYPE_F32, MX_DTYPE_BF16
_I32, _I8, _F32 = torch.int32, torch.int8, torch.float32


def _argtypes(lib):
    import ctypes

    P, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    lib.mx_route_rows.argtypes = [I64, I32, I32, I32]
    lib.mx_route_workspace.argtypes = [I64, I32]
    lib.i8_linear_workspace.argtypes = [I64, I64]
    for f in (lib.mx_route_rows, lib.mx_route_workspace, lib.i8_linear_workspace):
        f.restype = I64
    lib.mx_route.argtypes = [P, I32, I64, I32, I64, P, I32, I32, I32, I64, P, P, P, P, P, P, P, P, P, P, I64, P]
    lib.mx_route_grad.argtypes = [P, I32, I64, I32, I64, P, I32, I32, P, P, P, P, P, P, P, I64, P]
    lib.mx_dispatch.argtypes = [P, I32, I64, I64, I64, P, P, I32, I64, P, I64, P]
    lib.mx_dispatch_i8.argtypes = [P, I32, I64, I64, I64, P, P, I32, I64, P, I64, P, P]
    lib.i8_quantize_rows.argtypes = [P, I32, I64, I64, I64, P, I64, P, P]
    lib.i8_gemm_nt.argtypes = [P, I64, P, P, I64, P, P, I64, I64, I64, P, I64, I32, P]
    lib.i8_linear.argtypes = [P, I32, I64, P, I64, P, P, I64, I64, I64, P, I64, I32, P, I64, P]
    lib.i8_grouped_gemm_rows.argtypes = [P, I64, P, P, I64, I64, P, I64, P, I32, I64, I64, I64, P, I64, I32, P]
    lib.mx_combine.argtypes = [P, I32, I64, I64, I64, P, P, I32, I64, P, I64, P]
    lib.mx_combine_grad.argtypes = [P, I32, I64, I64, I64, P, I64, P, P, P, I32, I64, P, I64, P, P]
    F = ctypes.c_float
    lib.mx_route_scored.argtypes = [P, I32, I64, I32, I64, P, P, I32, I32, I32, I32, I32, I32, F, I32, I64, P, P, P, P, P,
                                    P, P, P, P, P, I64, P]
    lib.mx_route_scored_grad.argtypes = [P, I32, I64, I32, I64, P, I32, I32, I32, F, P, P, P, P, P, P, I64, P]
    lib.mx_route_bias_step.argtypes = [P, P, I32, F, P, P]
    for f in (lib.mx_route_scored, lib.mx_route_scored_grad, lib.mx_route_bias_step):
        f.restype = ctypes.c_int
    for f in (lib.mx_route, lib.mx_route_grad, lib.mx_dispatch, lib.mx_dispatch_i8, lib.i8_quantize_rows,
              lib.i8_gemm_nt, lib.i8_linear, lib.i8_grouped_gemm_rows, lib.mx_combine, lib.mx_combine_grad):
        f.restype = ctypes.c_int


_lib = None


def _L():
    global _lib
    if _lib is None:
        from . import library

        lib = library()
        _argtypes(lib)
        _lib = lib
    return _lib


# The current device's index and a device's current stream: torch's quickest
# ways, which are private, or its public ones where a torch has no such names.
_device = getattr(torch._C, "_cuda_getDevice", None) or (lambda: torch.cuda.current_device())
_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _run(i, f, *args):
    """Call an entry point on device i's current stream and raise on a status."""
    if i == _device():
        rc = f(*args, _stream(i))
    else:
        with torch.cuda.device(i):
            rc = f(*args, _stream(i))
    if rc:
        from . import MXError, status_string

        raise MXError(rc, status_string(rc))


# The checks below answer for a good argument at once; what is wrong with a bad
# one is found out apart, since the smallest calls last as long as their checks.
# Devices go by index: -1 is the host.
def _matrix(t, name, dtypes, i=None):
    """(row pitch, rows, cols) of a 2-d device tensor with contiguous rows."""
    try:
        rows, cols = t.shape
        pitch, step = t.stride()
        on = t.get_device()
        if (on == i if i is not None else on >= 0) and t.dtype in dtypes and (step == 1 or cols <= 1):
            if pitch >= cols:
                return pitch, rows, cols
            if rows <= 1:
                return cols, rows, cols
    except (AttributeError, TypeError, ValueError):
        pass
    _bad_matrix(t, name, dtypes, i)


def _bad_matrix(t, name, dtypes, i):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must have dtype {' or '.join(map(str, dtypes))}, not {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, not {tuple(t.shape)}")
    if i is not None and t.get_device() != i:
        raise ValueError(f"{name} is on {t.device}, the call runs on cuda:{i}")
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"{name} must have contiguous rows")
    raise ValueError(f"the rows of {name} must not overlap")


def _flat(t, name, dtype, shape, i):
    """A contiguous device tensor of one dtype and shape; returns its pointer."""
    if isinstance(t, torch.Tensor):
        if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == i:
            return t.data_ptr()
        if t.dtype is dtype and t.get_device() != i:
            raise ValueError(f"{name} is on {t.device}, the call runs on cuda:{i}")
        if t.dtype is dtype:
            raise ValueError(f"{name} must be contiguous with shape {tuple(shape)}, not {tuple(t.shape)}")
    raise ValueError(f"{name} must be a {dtype} tensor")


def _valid(valid, T, i):
    if valid is None:
        return None
    if valid.dtype is torch.bool:
        return _flat(valid, "valid", torch.bool, (T,), i)
    return _flat(valid, "valid", torch.uint8, (T,), i)


def _out_matrix(out, name, shape, dtype, like):
    """`out`, or a new matrix on the device of `like`; and its row pitch."""
    if out is None:
        return like.new_empty_strided(shape, (shape[1], 1), dtype=dtype), shape[1]   # the quickest of torch's ways
    pitch = _matrix(out, name, (dtype,), like.get_device())[0]
    if out.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(out.shape)}")
    return out, pitch


class MXRouting:
    """Outputs and workspace of mx_route and mx_route_scored for one (T, E, k,
    align), reused from call to call; made by mx_routing.

    idx, weight, slot [T, k]; src [rows]; counts, offs, prob [E]; live, loss
    [1]: see mx_route.  `normalize` is what the last call used, `scored` its
    (score, scale) or None where it was mx_route, `masked` whether it was given
    `valid`, `generation` how many have written here
    (replays of a captured graph are not counted): what needs the same routing
    later, a backward pass above all, notes the generation and hands it to
    mx_route_grad or `require`.  The tensors stay the plan's own: none can be
    put in another's place, and none may be resized."""

    __slots__ = ("T", "E", "k", "align", "rows", "device", "normalize", "masked", "generation", "scored", "idx", "weight", "slot",
                 "src", "counts", "offs", "live", "prob", "loss", "_workspace", "_ptrs")

    def __setattr__(self, name, value):
        if hasattr(self, "_ptrs") and name != "normalize":
            raise AttributeError(f"{name} of a routing cannot be replaced")
        object.__setattr__(self, name, value)

    def __init__(self, T, E, k, align, device):
        lib = _L()
        self.T, self.E, self.k, self.align = int(T), int(E), int(k), int(align)
        self.rows = lib.mx_route_rows(self.T, self.E, self.k, self.align)
        if self.rows < 0:
            raise ValueError(f"no routing of T={T}, E={E}, k={k}, align={align}: T >= 0, 1 <= E <= 1024, "
                             "1 <= k <= min(E, 16), 1 <= align <= 65536 and T k <= 2^30 are needed")
        dev = torch.device(device)
        if dev.type != "cuda":
            raise ValueError("device must be a GPU")
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device, self.normalize, self.masked, self.generation, self.scored = dev, True, False, 0, None
        e = lambda shape, dt: torch.empty(shape, dtype=dt, device=dev)  # noqa: E731
        self.idx, self.weight, self.slot = e((T, k), _I32), e((T, k), _F32), e((T, k), _I32)
        self.src, self.counts, self.offs = e((self.rows,), _I32), e((E,), _I32), e((E,), _I32)
        self.live, self.prob, self.loss = e((1,), _I32), e((E,), _F32), e((1,), _F32)
        size = lib.mx_route_workspace(self.T, self.E)
        self._workspace = e((size,), torch.uint8)
        self._ptrs = tuple(t.data_ptr() for t in (self.idx, self.weight, self.slot, self.src, self.counts, self.offs,
                                                  self.live, self.prob, self.loss, self._workspace)) + (size,)

    def record_stream(self, stream) -> None:
        """As a tensor's: before the routing is dropped, name every other stream
        that calls on it were made on, so that its memory (the workspace's too)
        is not handed out while they work."""
        for t in (self.idx, self.weight, self.slot, self.src, self.counts, self.offs, self.live, self.prob, self.loss,
                  self._workspace):
            t.record_stream(stream)

    def require(self, generation: int) -> None:
        """Raise unless this is still the routing of that generation."""
        if generation != self.generation:
            raise ValueError(f"the routing has been written again: generation {self.generation}, {generation} is needed "
                             "(passes that are alive at once need a routing each)")


# What a call leaves in a routing, past the guard above.
_set_normalize, _set_masked = MXRouting.normalize.__set__, MXRouting.masked.__set__
_set_generation, _set_scored = MXRouting.generation.__set__, MXRouting.scored.__set__


def _written(out, normalize, valid, scored):
    _set_normalize(out, bool(normalize))
    _set_masked(out, valid is not None)
    _set_scored(out, scored)
    _set_generation(out, out.generation + 1)
    return out


def mx_routing(T: int, E: int, k: int, align: int = 128, device="cuda") -> MXRouting:
    """The buffers of mx_route for T tokens, E experts and k picks each, groups
    padded to multiples of `align` (128 for the MXFP8 grouped calls).  Each
    mx_route writes them anew: streams that run at once, and forward passes
    whose backward is still to come, need a routing each.  The calls do not keep
    its memory: where another stream than the one it was made on works on it,
    hold the routing until that work is done, or record_stream it."""
    return MXRouting(T, E, k, align, device)


def mx_route(logits: torch.Tensor, k: int | None = None, valid: torch.Tensor | None = None, normalize: bool = True,
             align: int = 128, out: MXRouting | None = None) -> MXRouting:
    """Softmax routing of logits [T, E] (float32 or bfloat16, rows at any
    pitch) to the k best experts of each token.

    valid (bool or uint8 [T]) leaves tokens out, a logit of -inf an expert.
    The result's weight are the picks' probabilities, over their sum when
    `normalize`; counts, offs, slot and src describe the padded buffer that
    the grouped casts and products take; loss is the balance loss.  With out (an
    MXRouting) k and align are those it was made for."""
    ld, T, E = _matrix(logits, "logits", _ESZ)
    i = logits.get_device()
    out = _plan(out, logits, T, E, k, align)
    _run(i, _L().mx_route, logits.data_ptr(), _ESZ[logits.dtype], T, E, ld, _valid(valid, T, i), out.k,
         1 if normalize else 0, out.align, out.rows, *out._ptrs)
    return _written(out, normalize, valid, None)


SCORES = {"sigmoid": 0, "softmax": 1}


def mx_route_scored(logits: torch.Tensor, k: int | None = None, bias: torch.Tensor | None = None, score: str = "sigmoid",
                    groups: int = 1, top_groups: int | None = None, group_best: int = 2, normalize: bool = True,
                    scale: float = 1.0, valid: torch.Tensor | None = None, align: int = 128,
                    out: MXRouting | None = None) -> MXRouting:
    """Routing of logits [T, E] (float32 or bfloat16, rows at any pitch) by
    sigmoid or softmax scores s.

    The k experts of largest s + bias (float32 [E]; it decides picks alone) are
    taken out of the top_groups (None: all) of `groups` groups of neighbouring
    experts, those whose group_best (1 or 2) largest s + bias sum to most.  The
    result's weight are scale s of the picks, over their sum when `normalize`.
    valid, align, out and the rest of the result as for mx_route."""
    code = SCORES.get(score)
    if code is None:
        raise ValueError(f"score must be one of {', '.join(SCORES)}, not {score!r}")
    ld, T, E = _matrix(logits, "logits", _ESZ)
    i = logits.get_device()
    if top_groups is None:
        top_groups = groups
    if not 1 <= groups <= 32 or E % groups or not 1 <= top_groups <= groups or group_best not in (1, 2):
        raise ValueError(f"{groups} groups (top {top_groups}, best {group_best}) of E={E} experts: 1 to 32 groups of equal "
                         "size, 1 <= top_groups <= groups, group_best 1 or 2 are needed")
    b = None if bias is None else _flat(bias, "bias", _F32, (E,), i)
    v = _valid(valid, T, i)
    picks = out.k if out is not None else k
    if picks is not None and picks > top_groups * (E // groups):
        raise ValueError(f"k={picks} picks out of {top_groups} groups of {E // groups} experts")
    out = _plan(out, logits, T, E, k, align)
    _run(i, _L().mx_route_scored, logits.data_ptr(), _ESZ[logits.dtype], T, E, ld, v, b, code, groups, top_groups,
         group_best, out.k, 1 if normalize else 0, scale, out.align, out.rows, *out._ptrs)
    return _written(out, normalize, valid, (score, float(scale)))


def mx_route_scored_grad(logits: torch.Tensor, routing: MXRouting, dweight: torch.Tensor | None = None,
                         dloss: torch.Tensor | None = None, valid: torch.Tensor | None = None,
                         out: torch.Tensor | None = None, generation: int | None = None) -> torch.Tensor:
    """mx_route_grad of a routing that mx_route_scored wrote (its score, scale
    and normalize are the routing's)."""
    ld, T, E = _matrix(logits, "logits", _ESZ)
    i = logits.get_device()
    if routing.scored is None:
        raise ValueError("the routing was not written by mx_route_scored")
    dw, dl, v = _grad_inputs(routing, T, E, i, dweight, dloss, valid, generation)
    out, ld_d = _out_matrix(out, "out", (T, E), logits.dtype, logits)
    p = routing._ptrs
    score, scale = routing.scored
    _run(i, _L().mx_route_scored_grad, logits.data_ptr(), _ESZ[logits.dtype], T, E, ld, v, SCORES[score], routing.k,
         1 if routing.normalize else 0, scale, p[0], dw, p[4], p[6], dl, out.data_ptr(), ld_d)
    return out


def mx_route_bias_step(bias: torch.Tensor, counts: torch.Tensor, rate: float, out: torch.Tensor | None = None):
    """bias + rate sign(mean of counts - counts): float32 [E] for counts int32
    [E] of a routing (or their sums over ranks); out may be bias itself."""
    if not isinstance(bias, torch.Tensor) or not bias.is_cuda or bias.dim() != 1:
        raise ValueError("bias must be a float32 [E] device tensor")
    i, E = bias.get_device(), bias.shape[0]
    b, c = _flat(bias, "bias", _F32, (E,), i), _flat(counts, "counts", _I32, (E,), i)
    if out is None:
        out = bias.new_empty_strided((E,), (1,))
    _run(i, _L().mx_route_bias_step, b, c, E, rate, _flat(out, "out", _F32, (E,), i))
    return out


def _plan(out, logits, T, E, k, align):
    """`out`, checked against the call, or a new routing."""
    if out is None:
        if k is None:
            raise ValueError("k is needed when out is not given")
        return MXRouting(T, E, k, align, logits.device)
    if out.T != T or out.E != E or out.device.index != logits.get_device() or (k is not None and k != out.k):
        raise ValueError(f"out was made for T={out.T}, E={out.E}, k={out.k} on {out.device}, the call has T={T}, "
                         f"E={E}, k={k} on {logits.device}")
    return out


def _grad_inputs(routing, T, E, i, dweight, dloss, valid, generation):
    """Pointers of a routing gradient's inputs, checked against the routing."""
    if routing.T != T or routing.E != E or routing.device.index != i:
        raise ValueError("routing was made for other logits")
    if valid is None and routing.masked:
        raise ValueError("the routing was given valid, its gradient needs it too")
    if generation is not None:
        routing.require(generation)
    dw = None if dweight is None else _flat(dweight, "dweight", _F32, (T, routing.k), i)
    dl = None if dloss is None else _flat(dloss, "dloss", _F32, (1,), i)
    return dw, dl, _valid(valid, T, i)


def mx_route_grad(logits: torch.Tensor, routing: MXRouting, dweight: torch.Tensor | None = None,
                  dloss: torch.Tensor | None = None, valid: torch.Tensor | None = None,
                  out: torch.Tensor | None = None, generation: int | None = None) -> torch.Tensor:
    """Gradient of the routing's weight (dweight float32 [T, k]) and loss
    (dloss float32 [1]) with respect to the logits, in their dtype.  The routing
    does not keep its `valid`: a call without it is refused where mx_route had
    one, since the tokens it left out would get a gradient.  With `generation`
    (the routing's, noted after its mx_route) a routing that has been written
    since is refused."""
    ld, T, E = _matrix(logits, "logits", _ESZ)
    i = logits.get_device()
    if routing.scored is not None:
        raise ValueError("the routing was written by mx_route_scored: its gradient is mx_route_scored_grad")
    dw, dl, v = _grad_inputs(routing, T, E, i, dweight, dloss, valid, generation)
    out, ld_d = _out_matrix(out, "out", (T, E), logits.dtype, logits)
    p = routing._ptrs
    _run(i, _L().mx_route_grad, logits.data_ptr(), _ESZ[logits.dtype], T, E, ld, v, routing.k,
         1 if routing.normalize else 0, p[0], p[1], dw, p[4], p[6], dl, out.data_ptr(), ld_d)
    return out


def _slots(slot, i):
    """(pointer, T, k)"""
    try:
        T, k = slot.shape
        if slot.dtype is _I32 and slot.is_contiguous() and slot.get_device() == i:
            return slot.data_ptr(), T, k
    except (AttributeError, TypeError, ValueError):
        raise ValueError("slot must be an int32 [T, k] tensor") from None
    return _flat(slot, "slot", _I32, (T, k), i), T, k


def _src(src, i):
    """(pointer, M)"""
    try:
        (M,) = src.shape
        if src.dtype is _I32 and src.is_contiguous() and src.get_device() == i:
            return src.data_ptr(), M
    except (AttributeError, TypeError, ValueError):
        raise ValueError("src must be an int32 [M] tensor") from None
    return _flat(src, "src", _I32, (M,), i), M


def mx_dispatch(x: torch.Tensor, slot: torch.Tensor, src: torch.Tensor, out: torch.Tensor | None = None):
    """Rows of the padded buffer: x[t] at slot[t, j] for every pick, 0 where
    src is -1.  x is float32 or bfloat16 [T, N] with rows at any pitch."""
    ld, rows, N = _matrix(x, "x", _ESZ)
    i = x.get_device()
    sp, T, k = _slots(slot, i)
    rp, M = _src(src, i)
    if T != rows:
        raise ValueError(f"slot has {T} tokens, x {rows}")
    out, ld_o = _out_matrix(out, "out", (M, N), x.dtype, x)
    _run(i, _L().mx_dispatch, x.data_ptr(), _ESZ[x.dtype], T, N, ld, sp, rp, k, M, out.data_ptr(), ld_o)
    return out


def _codes_out(out, rows, K, like):
    """(q, its pitch, s): new codes get rows of whole 16-byte pieces, which the
    products read fastest."""
    if out is None:
        pitch = (K + 15) // 16 * 16
        return like.new_empty_strided((rows, K), (pitch, 1), dtype=_I8), pitch, like.new_empty_strided((rows,), (1,), dtype=_F32)
    q, s = out
    if q is None:
        raise ValueError("out must be two tensors, the codes and the scales")
    q, pitch = _out_matrix(q, "out[0]", (rows, K), _I8, like)
    _flat(s, "out[1]", _F32, (rows,), like.get_device())
    return q, pitch, s


def mx_dispatch_i8(x: torch.Tensor, slot: torch.Tensor, src: torch.Tensor, out=None):
    """mx_dispatch with each row quantized: (q int8 [M, K], s float32 [M])."""
    ld, rows, K = _matrix(x, "x", _ESZ)
    i = x.get_device()
    sp, T, k = _slots(slot, i)
    rp, M = _src(src, i)
    if T != rows:
        raise ValueError(f"slot has {T} tokens, x {rows}")
    q, pitch, s = _codes_out(out, M, K, x)
    _run(i, _L().mx_dispatch_i8, x.data_ptr(), _ESZ[x.dtype], T, K, ld, sp, rp, k, M, q.data_ptr(), pitch,
         s.data_ptr())
    return q, s


def i8_quantize_rows(x: torch.Tensor, out=None):
    """(q int8 [T, K], s float32 [T]): x[t] ~ q[t] s[t], s = max |x[t]| / 127."""
    ld, T, K = _matrix(x, "x", _ESZ)
    q, pitch, s = _codes_out(out, T, K, x)
    _run(x.get_device(), _L().i8_quantize_rows, x.data_ptr(), _ESZ[x.dtype], T, K, ld, q.data_ptr(), pitch, s.data_ptr())
    return q, s


def _bias(bias, N, i):
    return None if bias is None else _flat(bias, "bias", _F32, (N,), i)


def _product_out(out, shape, out_dtype, like):
    if out is None:
        if out_dtype not in _ESZ:
            raise ValueError(f"out_dtype must be float32 or bfloat16, not {out_dtype}")
        return like.new_empty_strided(shape, (shape[1], 1), dtype=out_dtype), shape[1]
    if out.dtype not in _ESZ:
        raise ValueError(f"out must be float32 or bfloat16, not {out.dtype}")
    return _out_matrix(out, "out", shape, out.dtype, like)


def i8_gemm_nt(A: torch.Tensor, sA: torch.Tensor, B: torch.Tensor, sB: torch.Tensor,
               bias: torch.Tensor | None = None, out_dtype=torch.bfloat16, out: torch.Tensor | None = None):
    """C = A B^T: int8 codes A [M, K] and B [N, K] (rows at any pitch), float32
    scales sA [M] and sB [N], optional float32 bias [N]."""
    lda, M, K = _matrix(A, "A", (_I8,))
    i = A.get_device()
    ldb, N, KB = _matrix(B, "B", (_I8,), i)
    if KB != K:
        raise ValueError("A and B must share the contraction extent")
    sa, sb, bi = _flat(sA, "sA", _F32, (M,), i), _flat(sB, "sB", _F32, (N,), i), _bias(bias, N, i)
    out, ldc = _product_out(out, (M, N), out_dtype, A)
    _run(i, _L().i8_gemm_nt, A.data_ptr(), lda, sa, B.data_ptr(), ldb, sb, bi, M, N, K, out.data_ptr(), ldc,
         _ESZ[out.dtype])
    return out


def i8_linear(x: torch.Tensor, B: torch.Tensor, sB: torch.Tensor, bias: torch.Tensor | None = None, out_dtype=None,
              out: torch.Tensor | None = None):
    """i8_quantize_rows of x [M, K] and i8_gemm_nt in one call; the result has
    x's dtype unless out_dtype or out says otherwise."""
    ld, M, K = _matrix(x, "x", _ESZ)
    i = x.get_device()
    ldb, N, KB = _matrix(B, "B", (_I8,), i)
    if KB != K:
        raise ValueError("x and B must share the contraction extent")
    sb, bi = _flat(sB, "sB", _F32, (N,), i), _bias(bias, N, i)
    out, ldc = _product_out(out, (M, N), out_dtype or x.dtype, x)
    size = M * ((K + 15) // 16 * 16) + (M * 4 + 15) // 16 * 16
    ws = x.new_empty_strided((size,), (1,), dtype=torch.uint8)
    _run(i, _L().i8_linear, x.data_ptr(), _ESZ[x.dtype], ld, B.data_ptr(), ldb, sb, bi, M, N, K, out.data_ptr(), ldc,
         _ESZ[out.dtype], ws.data_ptr(), size)
    return out


def i8_grouped_gemm_rows(A: torch.Tensor, sA: torch.Tensor, B: torch.Tensor, sB: torch.Tensor, offs: torch.Tensor,
                         out_dtype=torch.bfloat16, out: torch.Tensor | None = None):
    """Rows of group g (cumulative int32 ends offs [G], groups of any size) with
    expert g's codes B[g] ([E, N, K], E >= G) and scales sB[g] ([E, N]); rows
    from offs[-1] on give 0."""
    lda, M, K = _matrix(A, "A", (_I8,))
    i = A.get_device()
    if not isinstance(B, torch.Tensor) or B.dtype is not _I8 or B.dim() != 3 or B.get_device() != i:
        raise ValueError("B must be int8 [E, N, K] codes on the device of A")
    E, N, KB = B.shape
    b_gs, ldb, step = B.stride()
    if KB != K or (K > 1 and step != 1) or (N > 1 and ldb < K):
        raise ValueError("B must be [E, N, K] codes with contiguous rows that share A's contraction extent")
    if not isinstance(sB, torch.Tensor) or sB.dtype is not _F32 or sB.shape != (E, N) or sB.get_device() != i or (
            N > 1 and sB.stride(1) != 1):
        raise ValueError("sB must be a float32 [E, N] tensor with contiguous rows")
    if not isinstance(offs, torch.Tensor) or offs.dim() != 1 or not 1 <= offs.shape[0] <= E:
        raise ValueError("offs must be an int32 [G] tensor with 1 <= G <= E")
    G = offs.shape[0]
    sa, of = _flat(sA, "sA", _F32, (M,), i), _flat(offs, "offs", _I32, (G,), i)
    out, ldc = _product_out(out, (M, N), out_dtype, A)
    _run(i, _L().i8_grouped_gemm_rows, A.data_ptr(), lda, sa, B.data_ptr(), ldb if ldb > K else K, b_gs,
         sB.data_ptr(), sB.stride(0), of, G, M, N, K, out.data_ptr(), ldc, _ESZ[out.dtype])
    return out


def mx_combine(rows: torch.Tensor, slot: torch.Tensor, weight: torch.Tensor | None = None,
               out: torch.Tensor | None = None):
    """y[t] = sum_j weight[t, j] rows[slot[t, j]] (weight None: 1) over the
    picks that have a slot."""
    ld, M, N = _matrix(rows, "rows", _ESZ)
    i = rows.get_device()
    sp, T, k = _slots(slot, i)
    wp = None if weight is None else _flat(weight, "weight", _F32, (T, k), i)
    out, ld_y = _out_matrix(out, "out", (T, N), rows.dtype, rows)
    _run(i, _L().mx_combine, rows.data_ptr(), _ESZ[rows.dtype], M, N, ld, sp, wp, k, T, out.data_ptr(), ld_y)
    return out


def mx_combine_grad(dy: torch.Tensor, rows: torch.Tensor, slot: torch.Tensor, weight: torch.Tensor | None,
                    src: torch.Tensor, out=None):
    """(drows, dweight) of mx_combine for dy [T, N]: drows[slot[t, j]] =
    weight[t, j] dy[t], 0 where src is -1; dweight[t, j] = <dy[t],
    rows[slot[t, j]]>."""
    ld_g, tokens, N = _matrix(dy, "dy", _ESZ)
    i = dy.get_device()
    ld_r = _matrix(rows, "rows", (dy.dtype,), i)[0]
    sp, T, k = _slots(slot, i)
    rp, M = _src(src, i)
    if tokens != T or rows.shape != (M, N):
        raise ValueError(f"dy must be [{T}, N] and rows [{M}, N], not {tuple(dy.shape)} and {tuple(rows.shape)}")
    wp = None if weight is None else _flat(weight, "weight", _F32, (T, k), i)
    drows, dweight = out if out is not None else (None, None)
    drows, ld_d = _out_matrix(drows, "out[0]", (M, N), dy.dtype, dy)
    if dweight is None:
        dweight = dy.new_empty_strided((T, k), (k, 1), dtype=_F32)
    dp = _flat(dweight, "out[1]", _F32, (T, k), i)
    _run(i, _L().mx_combine_grad, dy.data_ptr(), _ESZ[dy.dtype], T, N, ld_g, rows.data_ptr(), ld_r, sp, wp, rp, k, M,
         drows.data_ptr(), ld_d, dp)
    return drows, dweight
