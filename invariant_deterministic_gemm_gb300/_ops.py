"""Python binding of the mixture-of-experts operators (include/det_ops.h).

Argument marshalling only, in the manner of the det_gemm binding: every
function takes CUDA tensors, checks their types and layouts, allocates what
is not given with PyTorch (on the stream the work runs on) and calls the C
function of the same name. There is no fallback.

  det_moe_route(logits, top_k, ...)               -> weights, ids
  det_moe_route_bwd(dweights, logits, ids, ...)   -> dlogits
  det_moe_dispatch(ids, num_experts)              -> offsets, rows, slots
  det_moe_gather(x, rows, top_k)                  -> xs      (gradient: det_moe_combine)
  det_moe_combine(ys, slots, weights=None)        -> y
  det_moe_combine_bwd(dy, ys, rows, slots, weights) -> dys, dweights
  det_fp8_quantize_rows(x, rows=None, top_k=1)    -> q, scales
  det_fp8_quantize_cols(x, offsets=None)          -> qt, scales
  det_fp8_quantize_tiles(w, transposed=False)     -> q, scales
  det_fp8_gemm(A, sa, W, sw)                      -> C
  det_fp8_gemm_grouped(A, sa, W, sw, offsets)     -> C
  det_fp8_gemm_wgrad(Yt, sy, Xt, sx, offsets)     -> dW
  det_embedding(tokens, table, scale)             -> out
  det_embedding_grad(dy, tokens, vocab, scale)    -> dtable
"""
from __future__ import annotations

import ctypes

import torch

import invariant_deterministic_gemm_gb300 as _dg

BLOCK = 128
MAX_EXPERTS = 512
MAX_TOP_K = 32
_BF16, _F32, _I32, _E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn
_SCORES = {"softmax": 0, "sigmoid": 1}

_p, _i, _q, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
_SIGNATURES = {
    "det_moe_route": [_p, _i, _p, _p, _p, _q, _q, _q, _i, _i, _i, _i, _i, _i, _f, _p],
    "det_moe_route_bwd": [_p, _p, _i, _p, _p, _q, _q, _q, _q, _i, _i, _i, _f, _p],
    "det_moe_dispatch": [_p, _p, _p, _p, _q, _q, _i, _p],
    "det_moe_gather": [_p, _p, _p, _q, _q, _q, _i, _q, _q, _p],
    "det_moe_combine": [_p, _p, _p, _p, _q, _q, _q, _i, _q, _q, _p],
    "det_moe_combine_bwd": [_p, _p, _p, _p, _p, _p, _p, _q, _q, _i, _q, _q, _q, _p],
    "det_fp8_quantize_rows": [_p, _p, _p, _p, _q, _q, _q, _i, _q, _q, _q, _p],
    "det_fp8_quantize_cols": [_p, _p, _p, _p, _q, _q, _q, _q, _q, _q, _q, _p],
    "det_fp8_quantize_tiles": [_p, _p, _p, _p, _p, _q, _q, _q, _q, _q, _q, _q, _q, _q, _p],
    "det_fp8_gemm": [_p, _p, _p, _p, _p, _i, _q, _q, _q, _q, _q, _q, _q, _q, _q, _p],
    "det_fp8_gemm_grouped": [_p, _p, _p, _p, _p, _p, _i] + [_q] * 12 + [_p],
    "det_fp8_gemm_wgrad": [_p, _p, _p, _p, _p, _p, _i] + [_q] * 11 + [_p],
    "det_embedding": [_p, _i, _p, _p, _q, _q, _q, _f, _q, _q, _p],
    "det_embedding_grad": [_p, _p, _i, _p, _i, _q, _q, _q, _f, _q, _i, _q, _q, _p, _q, _p],
    "det_embedding_grad_workspace": [_q, _q, _q],
    "det_ops_check": [_p],
    "det_ops_debug_force_timeout": [_i],
}
_fns = {}


def _fn(name):
    fn = _fns.get(name)
    if fn is None:
        fn = getattr(_dg.lib(), name)
        fn.argtypes = _SIGNATURES[name]
        fn.restype = ctypes.c_int64 if name == "det_embedding_grad_workspace" else ctypes.c_int
        _fns[name] = fn
    return fn


def _run(name, *args):
    fn = _fns.get(name) or _fn(name)
    st = fn(*args)
    if st != 0:
        raise _dg.DetGemmError(st, name)


# A decode-sized call is bound by this module's own time, so each property of
# a tensor is read once, checks are one expression where they can be, and
# error messages are formatted only for an error.

def _on(stream, make, *args):
    """make(*args), its allocations belonging to the stream that uses them."""
    if stream is None:
        return make(*args)
    with torch.cuda.stream(stream):
        return make(*args)


def _flat(t, name, dtype, shape):
    """Data pointer of a contiguous tensor of one type and shape."""
    if isinstance(t, torch.Tensor) and t.dtype == dtype and t.is_cuda and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    raise ValueError("%s must be contiguous" % name)


_ELEM = {_BF16: 2, _F32: 4, _E4M3: 1}


def _mat(t, name, dtype):
    """(pointer, leading dimension, rows, columns) of a row-major CUDA matrix."""
    if isinstance(t, torch.Tensor) and t.dtype == dtype and t.is_cuda:
        shape = t.shape
        if len(shape) == 2:
            rows, cols = shape
            s0, s1 = t.stride()
            if s1 == 1 and rows > 1:
                return t.data_ptr(), s0, rows, cols
            p, ld = _dg._mat(t, name, dtype)
            return p, ld, rows, cols
    _dg._mat(t, name, dtype)
    raise AssertionError("unreachable")


def _mats(t, name, dtype):
    """(pointer, matrices, rows, cols, pitch, distance) of a [G, rows, cols] stack of row-major matrices."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    shape = t.shape
    if len(shape) != 3:
        raise ValueError("%s must be 3-D, got shape %s" % (name, tuple(shape)))
    G, rows, cols = shape
    gap, ld, s2 = t.stride()
    if G > 0 and rows > 1 and s2 == 1 and t.is_cuda:
        return t.data_ptr(), G, rows, cols, ld, gap if G > 1 else rows * ld
    per16 = 16 // _ELEM[dtype]
    if G and rows and cols:
        p, ld = _dg._mat(t[0], name, dtype)
    else:
        p, ld = t.data_ptr(), max(per16, (cols + per16 - 1) // per16 * per16)
    return p, G, rows, cols, ld, gap if G > 1 and rows and cols else rows * ld


def _new(rows, cols, dtype, device, mats=None):
    """A [rows, cols] (or [mats, rows, cols]) tensor with 16-byte row pitches."""
    per16 = 16 // _ELEM[dtype]
    ld = max(per16, (cols + per16 - 1) // per16 * per16)
    t = torch.empty((rows, ld) if mats is None else (mats, rows, ld), dtype=dtype, device=device)
    return t if ld == cols else t[..., :cols]


def _out(out, rows, cols, dtype, device, stream):
    """(out, pointer, pitch): the given output, or a new one."""
    if out is None:
        out = _new(rows, cols, dtype, device) if stream is None else _on(stream, _new, rows, cols, dtype, device)
        ld = out.stride(0)
        return out, out.data_ptr(), ld if ld else max(cols, 1)
    if tuple(out.shape) != (rows, cols):
        raise ValueError("out must have shape %s, got %s" % ((rows, cols), tuple(out.shape)))
    p, ld, _, _ = _mat(out, "out", dtype)
    return out, p, ld


def _score(score):
    if score not in _SCORES:
        raise ValueError("score must be 'softmax' or 'sigmoid', got %r" % (score,))
    return _SCORES[score]


def _logits(t, name="logits"):
    """(pointer, pitch, tokens, experts, is FP32) of a row-major matrix of logits."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    dtype = t.dtype
    if dtype != _F32 and dtype != _BF16:
        raise TypeError("%s must be torch.float32 or torch.bfloat16, got %s" % (name, dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    shape = t.shape
    if len(shape) != 2:
        raise ValueError("%s must be 2-D, got shape %s" % (name, tuple(shape)))
    T, E = shape
    s0, s1 = t.stride()
    if s1 != 1 and E > 1:
        raise ValueError("%s must be row-major with unit column stride" % name)
    return t.data_ptr(), s0 if T > 1 else max(E, s0), T, E, 1 if dtype == _F32 else 0


def _route_out(T, k, device):
    return torch.empty((T, k), dtype=_F32, device=device), torch.empty((T, k), dtype=_I32, device=device)


def det_moe_route(logits, top_k, *, score="softmax", bias=None, n_groups=1, top_groups=1, group_best=2,
                  renormalize=True, scale=1.0, stream=None):
    """The top_k experts of every token and their weights.

    logits [T, E] FP32 or BF16; bias [E] FP32 is added to the scores for the
    choice only. With n_groups > 1 only experts of the best top_groups groups
    are taken, a group's value being the sum of its best group_best choices.
    Returns weights [T, top_k] FP32 and ids [T, top_k] int32, best first, ties
    to the lower index. Experts with a logit of -inf or NaN are masked; a
    choice left over has id -1 and weight 0."""
    p, ld, T, E, fp32 = _logits(logits)
    b = None if bias is None else _flat(bias, "bias", _F32, (E,))
    weights, ids = _on(stream, _route_out, T, top_k, logits.device)
    _run("det_moe_route", p, fp32, b, weights.data_ptr(), ids.data_ptr(), T, E, ld, top_k, _score(score), n_groups,
         top_groups, group_best, 1 if renormalize else 0, scale, _dg._stream_handle(stream))
    return weights, ids


def det_moe_route_bwd(dweights, logits, ids, *, score="softmax", renormalize=True, scale=1.0, stream=None):
    """dlogits [T, E] (the logits' type) from dweights [T, top_k] FP32."""
    p, ld, T, E, fp32 = _logits(logits)
    i, n, k = _index2(ids, "ids")
    if n != T:
        raise ValueError("logits and ids disagree on the tokens: %d vs %d" % (T, n))
    d = _flat(dweights, "dweights", _F32, (T, k))
    out = _on(stream, _empty2, T, E, logits.dtype, logits.device)
    _run("det_moe_route_bwd", d, p, fp32, i, out.data_ptr(), T, E, ld, E, k, _score(score), 1 if renormalize else 0,
         scale, _dg._stream_handle(stream))
    return out


def _empty2(rows, cols, dtype, device):
    return torch.empty((rows, cols), dtype=dtype, device=device)


def _dispatch_out(E, T, k, device):
    return (torch.empty(E + 1 if E >= 0 else 0, dtype=_I32, device=device), torch.empty(T * k, dtype=_I32, device=device),
            torch.empty((T, k), dtype=_I32, device=device))


def det_moe_dispatch(ids, num_experts, *, stream=None):
    """Rows of the experts: ids [T, k] int32 -> offsets [E + 1], rows [T * k]
    (the pair t * k + j of each row, -1 past offsets[E]) and slots [T, k] (the
    row of each pair, -1 for an id outside [0, E)), all int32 on the device."""
    p, T, k = _index2(ids, "ids")
    offsets, rows, slots = _on(stream, _dispatch_out, num_experts, T, k, ids.device)
    _run("det_moe_dispatch", p, offsets.data_ptr(), rows.data_ptr(), slots.data_ptr(), T, num_experts, k,
         _dg._stream_handle(stream))
    return offsets, rows, slots


def _index1(t, name):
    """(pointer, length) of a contiguous int32 vector."""
    if isinstance(t, torch.Tensor):
        shape = t.shape
        if len(shape) == 1:
            return _flat(t, name, _I32, shape), shape[0]
    raise ValueError("%s must be a 1-D tensor" % name)


def _index2(t, name):
    """(pointer, rows, columns) of a contiguous int32 matrix."""
    if isinstance(t, torch.Tensor):
        shape = t.shape
        if len(shape) == 2:
            return _flat(t, name, _I32, shape), shape[0], shape[1]
    raise ValueError("%s must be a 2-D tensor" % name)


def det_moe_gather(x, rows, top_k, *, out=None, stream=None):
    """xs[r] = x[rows[r] // top_k] (zero where rows[r] < 0), BF16. Its
    gradient is det_moe_combine(dxs, slots)."""
    p, ld, T, H = _mat(x, "x", _BF16)
    r, R = _index1(rows, "rows")
    out, o, ldo = _out(out, R, H, _BF16, x.device, stream)
    _run("det_moe_gather", p, r, o, T, R, H, top_k, ld, ldo, _dg._stream_handle(stream))
    return out


def det_moe_combine(ys, slots, weights=None, *, out=None, stream=None):
    """y[t] = sum over j of weights[t, j] * ys[slots[t, j]] (weights None: 1),
    in FP32 in ascending j, rounded once to BF16."""
    p, ld, R, H = _mat(ys, "ys", _BF16)
    s, T, k = _index2(slots, "slots")
    w = None if weights is None else _flat(weights, "weights", _F32, (T, k))
    out, o, ldo = _out(out, T, H, _BF16, ys.device, stream)
    _run("det_moe_combine", p, s, w, o, T, R, H, k, ld, ldo, _dg._stream_handle(stream))
    return out


def _combine_bwd_out(T, k, H, device):
    return _new(T * k, H, _BF16, device), torch.empty((T, k), dtype=_F32, device=device)


def det_moe_combine_bwd(dy, ys, rows, slots, weights, *, stream=None):
    """Gradients of det_moe_combine: dys [T * k, H] BF16 and dweights [T, k] FP32."""
    g, ldg, T, H = _mat(dy, "dy", _BF16)
    s, n, k = _index2(slots, "slots")
    if n != T:
        raise ValueError("dy and slots disagree on the tokens: %d vs %d" % (T, n))
    r = _flat(rows, "rows", _I32, (T * k,))
    w = _flat(weights, "weights", _F32, (T, k))
    y, ldy, R, H2 = _mat(ys, "ys", _BF16)
    if R != T * k or H2 != H:
        raise ValueError("ys must have shape %s, got %s" % ((T * k, H), (R, H2)))
    dys, dw = _on(stream, _combine_bwd_out, T, k, H, dy.device)
    _run("det_moe_combine_bwd", g, y, r, s, w, dys.data_ptr(), dw.data_ptr(), T, H, k, ldg, ldy,
         dys.stride(0) or max(H, 1), _dg._stream_handle(stream))
    return dys, dw


def _rows_out(M, K, nb, device):
    return _new(M, K, _E4M3, device), torch.empty_strided((M, nb), (1, max(M, 1)), dtype=_F32, device=device)


def det_fp8_quantize_rows(x, rows=None, top_k=1, *, stream=None):
    """x [T, K] BF16 -> e4m3 [M, K] and one FP32 scale for each row and block
    of 128 columns, a [M, ceil(K / 128)] tensor stored block by block. With
    rows (det_moe_dispatch's) row r is x[rows[r] // top_k]: gather and
    quantise."""
    p, ld, T, K = _mat(x, "x", _BF16)
    r, M = (None, T) if rows is None else _index1(rows, "rows")
    q, s = _on(stream, _rows_out, M, K, (K + 127) // 128, x.device)
    _run("det_fp8_quantize_rows", p, r, q.data_ptr(), s.data_ptr(), T, M, K, top_k, ld, q.stride(0) or 16, M or 1,
         _dg._stream_handle(stream))
    return q, s


def _cols_out(K, nb, device):
    return torch.empty((K, nb * BLOCK), dtype=_E4M3, device=device), _new(nb, K, _F32, device)


def det_fp8_quantize_cols(x, offsets=None, *, stream=None):
    """x [M, K] BF16 -> its transpose in e4m3, [K, blocks * 128], and one FP32
    scale for each column of x and block of 128 rows, [blocks, K]. With offsets
    [G + 1] each group's rows form blocks of their own."""
    p, ld, M, K = _mat(x, "x", _BF16)
    o, G = (None, 0) if offsets is None else _index1(offsets, "offsets")
    G = max(G - 1, 0)
    nb = (M + 127) // 128 + G
    q, s = _on(stream, _cols_out, K, nb, x.device)
    _run("det_fp8_quantize_cols", p, o, q.data_ptr(), s.data_ptr(), M, K, G, nb, ld, nb * BLOCK, max(s.stride(0), 4),
         _dg._stream_handle(stream))
    return q, s


def _tiles_out(G, N, K, rt, ct, device):
    return _new(N, K, _E4M3, device, G), torch.empty((G, rt, ct), dtype=_F32, device=device)


def det_fp8_quantize_tiles(w, transposed=False, *, stream=None):
    """A weight [N, K] (or a stack [G, N, K]) BF16 -> e4m3 of its shape and one
    FP32 scale for each 128 x 128 tile. transposed: the quantised transpose
    [.., K, N] and its scales instead (the input gradient's operand)."""
    if not isinstance(w, torch.Tensor) or w.dim() not in (2, 3):
        raise ValueError("w must be a 2-D or 3-D tensor")
    flat = w.dim() == 2
    p, G, N, K, ld, gap = _mats(w[None] if flat else w, "w", _BF16)
    if not w.is_cuda:
        raise ValueError("w must be a CUDA tensor")
    rt, ct = _nblk(N), _nblk(K)
    q, s = _on(stream, _tiles_out, G, *((K, N, ct, rt) if transposed else (N, K, rt, ct)), w.device)
    a = (q.data_ptr(), s.data_ptr())
    args = (None, None) + a if transposed else a + (None, None)
    ldq, gq = max(q.stride(1), 16), max(q.stride(0), 16)
    _run("det_fp8_quantize_tiles", p, *args, G, N, K, ld, gap, ldq, gq, ldq, gq, _dg._stream_handle(stream))
    return (q[0], s[0]) if flat else (q, s)


_OUT_TYPES = {_BF16: 0, _F32: 1}


def _out_type(out_dtype):
    f = _OUT_TYPES.get(out_dtype)
    if f is None:
        raise TypeError("out_dtype must be torch.bfloat16 or torch.float32, got %s" % (out_dtype,))
    return f


def _row_scales(t, name, rows, blocks):
    if not isinstance(t, torch.Tensor) or t.dtype != _F32 or not t.is_cuda:
        raise TypeError("%s must be a float32 CUDA tensor" % name)
    if t.shape != (rows, blocks):
        raise ValueError("%s must have shape %s, got %s" % (name, (rows, blocks), tuple(t.shape)))
    s0, s1 = t.stride()
    return t.data_ptr(), s0, s1


def _tile_scales(t, name, shape):
    if not isinstance(t, torch.Tensor) or t.dtype != _F32 or not t.is_cuda:
        raise TypeError("%s must be a float32 CUDA tensor" % name)
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, shape, tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _nblk(n):
    return (n + 127) // 128


def det_fp8_gemm(A, a_scale, W, w_scale, *, out_dtype=_BF16, out=None, stream=None):
    """C[M, N] = dequantised A[M, K] @ dequantised W[N, K]^T. A and a_scale
    from det_fp8_quantize_rows, W and w_scale from det_fp8_quantize_tiles. The
    input gradient is det_fp8_gemm(dY, ..) with the transposed weight."""
    a, lda, M, K = _mat(A, "A", _E4M3)
    w, ldw, N, K2 = _mat(W, "W", _E4M3)
    if K2 != K:
        raise ValueError("inner dimensions differ: %d vs %d" % (K, K2))
    kb = (K + 127) // 128
    sa, sr, sb = _row_scales(a_scale, "a_scale", M, kb)
    ws = _tile_scales(w_scale, "w_scale", ((N + 127) // 128, kb))
    if out is not None:
        out_dtype = out.dtype
    f32 = _out_type(out_dtype)
    C, c, ldc = _out(out, M, N, out_dtype, A.device, stream)
    _run("det_fp8_gemm", a, sa, w, ws, c, f32, M, N, K, lda, sr, sb, ldw, kb, ldc, _dg._stream_handle(stream))
    return C


def det_fp8_gemm_grouped(A, a_scale, W, w_scale, offsets, *, out_dtype=_BF16, out=None, stream=None):
    """Rows [offsets[g], offsets[g+1]) of A [M, K] with expert g's weight of W
    [G, N, K] -> C [M, N]. offsets [G + 1] int32 stays on the device; rows
    outside every group become zero."""
    a, lda, M, K = _mat(A, "A", _E4M3)
    w, G, N, K2, ldw, gw = _mats(W, "W", _E4M3)
    if K2 != K:
        raise ValueError("inner dimensions differ: %d vs %d" % (K, K2))
    off = _flat(offsets, "offsets", _I32, (G + 1,))
    kb, nb = (K + 127) // 128, (N + 127) // 128
    sa, sr, sb = _row_scales(a_scale, "a_scale", M, kb)
    ws = _tile_scales(w_scale, "w_scale", (G, nb, kb))
    if out is not None:
        out_dtype = out.dtype
    f32 = _out_type(out_dtype)
    C, c, ldc = _out(out, M, N, out_dtype, A.device, stream)
    _run("det_fp8_gemm_grouped", a, sa, w, ws, off, c, f32, G, M, N, K, lda, sr, sb, ldw, gw, kb, nb * kb, ldc,
         _dg._stream_handle(stream))
    return C


def det_fp8_gemm_wgrad(Yt, y_scale, Xt, x_scale, offsets=None, *, out_dtype=_F32, out=None, stream=None):
    """dW[N, K] = dY^T X from det_fp8_quantize_cols of dY and of X (with the
    same offsets). With offsets [G + 1]: dW [G, N, K], one matrix an expert."""
    y, ldy, N, L = _mat(Yt, "Yt", _E4M3)
    x, ldx, K, L2 = _mat(Xt, "Xt", _E4M3)
    if L2 != L or L % BLOCK:
        raise ValueError("Yt and Xt must have the same whole number of blocks: %d vs %d columns" % (L, L2))
    nb = L // BLOCK
    sy, ldsy, b1, n1 = _mat(y_scale, "y_scale", _F32)
    sx, ldsx, b2, n2 = _mat(x_scale, "x_scale", _F32)
    if (b1, n1, b2, n2) != (nb, N, nb, K):
        raise ValueError("y_scale and x_scale must have shapes %s and %s, got %s and %s"
                         % ((nb, N), (nb, K), (b1, n1), (b2, n2)))
    G = 1
    off = None
    M = L
    if offsets is not None:
        off, G = _index1(offsets, "offsets")
        G -= 1
        M = (nb - G) * BLOCK                          # at least the tokens' number
        if G < 0 or M < 0:
            raise ValueError("offsets does not match the blocks of Yt and Xt")
    if out is not None:
        out_dtype = out.dtype
    f32 = _out_type(out_dtype)
    if out is None:
        out = _on(stream, _new, N, K, out_dtype, Yt.device, None if offsets is None else G)
    elif tuple(out.shape) != ((N, K) if offsets is None else (G, N, K)):
        raise ValueError("out must have shape %s, got %s" % ((N, K) if offsets is None else (G, N, K), tuple(out.shape)))
    if offsets is None:
        d, ldd, _, _ = _mat(out, "out", out_dtype)
        gd = 0
    else:
        d, _, _, _, ldd, gd = _mats(out, "out", out_dtype)
    _run("det_fp8_gemm_wgrad", y, sy, x, sx, off, d, f32, G, M, N, K, nb, max(ldy, 16), max(ldsy, 4), max(ldx, 16),
         max(ldsx, 4), ldd, gd, _dg._stream_handle(stream))
    return out


def _tokens(t):
    """(pointer, is int64, number) of a contiguous vector of tokens."""
    if not isinstance(t, torch.Tensor) or (t.dtype != torch.int64 and t.dtype != _I32):
        raise TypeError("tokens must be an int64 or int32 tensor")
    shape = t.shape
    if len(shape) != 1:
        raise ValueError("tokens must be 1-D, got shape %s" % (tuple(shape),))
    return _flat(t, "tokens", t.dtype, shape), 1 if t.dtype == torch.int64 else 0, shape[0]


def det_embedding(tokens, table, scale=1.0, *, out=None, stream=None):
    """out[t] = scale * table[tokens[t]], rounded once to BF16. A token outside
    the table gives a zero row and an error from det_gemm_check."""
    t, is64, T = _tokens(tokens)
    w, ld, V, H = _mat(table, "table", _BF16)
    out, o, ldo = _out(out, T, H, _BF16, table.device, stream)
    _run("det_embedding", t, is64, w, o, T, V, H, scale, ld, ldo, _dg._stream_handle(stream))
    return out


def _workspace(size, device):
    return torch.empty(max(size, 256), dtype=torch.uint8, device=device)


def det_embedding_grad(dy, tokens, vocab, scale=1.0, *, padding_idx=None, out_dtype=_F32, out=None, accumulate=False,
                       stream=None):
    """dtable[v] = scale * sum of dy[t] over tokens[t] == v, in a fixed order.
    With accumulate it is added to `out`; rows that never occur are then left
    alone, and become zero otherwise. padding_idx gets no gradient."""
    t, is64, n = _tokens(tokens)
    g, ldg, T, H = _mat(dy, "dy", _BF16)
    if n != T:
        raise ValueError("dy and tokens disagree on the tokens: %d vs %d" % (T, n))
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    if padding_idx is not None and not 0 <= padding_idx < vocab:
        raise ValueError("padding_idx must be in [0, vocab)")
    if out is not None:
        out_dtype = out.dtype
    f32 = _out_type(out_dtype)
    ws = _on(stream, _workspace, _fn("det_embedding_grad_workspace")(T, vocab, H), dy.device)
    out, o, ldo = _out(out, vocab, H, out_dtype, dy.device, stream)
    _run("det_embedding_grad", g, t, is64, o, f32, T, vocab, H, scale, -1 if padding_idx is None else padding_idx,
         1 if accumulate else 0, ldg, ldo, ws.data_ptr(), ws.numel(), _dg._stream_handle(stream))
    return out


def det_ops_check(stream=None) -> int:
    """Synchronise the stream and return (and clear) these operators' device status."""
    return int(_fn("det_ops_check")(_dg._stream_handle(stream)))


def det_ops_debug_force_timeout(enable: bool) -> None:
    """Test hook: make every later 8-bit product time out on purpose (see det_ops.h)."""
    _fn("det_ops_debug_force_timeout")(1 if enable else 0)


__all__ = [
    "det_moe_route", "det_moe_route_bwd", "det_moe_dispatch", "det_moe_gather", "det_moe_combine",
    "det_moe_combine_bwd", "det_fp8_quantize_rows", "det_fp8_quantize_cols", "det_fp8_quantize_tiles",
    "det_fp8_gemm", "det_fp8_gemm_grouped", "det_fp8_gemm_wgrad", "det_embedding", "det_embedding_grad",
    "det_ops_check", "det_ops_debug_force_timeout",
]
