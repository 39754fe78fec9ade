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

import contextlib
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
    st = _fn(name)(*args)
    if st != _dg.OK:
        raise _dg.DetGemmError(st, name)


def _on(stream):
    """Outputs and workspaces are allocated on the stream that uses them."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _flat(t, name, dtype, shape):
    """Data pointer of a contiguous tensor of one type and shape."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _mat(t, name, dtype):
    return _dg._mat(t, name, dtype)


def _mats(t, name, dtype):
    """(pointer, matrices, rows, cols, pitch, distance) of a [G, rows, cols] stack of row-major matrices."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dim() != 3:
        raise ValueError("%s must be 3-D, got shape %s" % (name, tuple(t.shape)))
    G, rows, cols = t.shape
    per16 = 16 // t.element_size()
    if G and rows and cols:
        p, ld = _mat(t[0], name, dtype)
        if t.dtype != dtype:
            raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
        gap = t.stride(0) if G > 1 else rows * ld
    else:
        if t.dtype != dtype:
            raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
        p, ld = t.data_ptr(), max(per16, (cols + per16 - 1) // per16 * per16)
        gap = rows * ld
    return p, G, rows, cols, ld, gap


def _new(rows, cols, dtype, device, mats=None):
    """A [rows, cols] (or [mats, rows, cols]) tensor with 16-byte row pitches."""
    size = 1 if dtype == _E4M3 else dtype.itemsize
    per16 = 16 // size
    ld = max(per16, (cols + per16 - 1) // per16 * per16)
    shape = (rows, ld) if mats is None else (mats, rows, ld)
    t = torch.empty(shape, dtype=dtype, device=device)
    return t if ld == cols else t[..., :cols]


def _given(out, shape, name="out"):
    if tuple(out.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(out.shape)))
    return out


def _score(score):
    if score not in _SCORES:
        raise ValueError("score must be 'softmax' or 'sigmoid', got %r" % (score,))
    return _SCORES[score]


def _logits(t, name="logits"):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype not in (_F32, _BF16):
        raise TypeError("%s must be torch.float32 or torch.bfloat16, got %s" % (name, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dim() != 2:
        raise ValueError("%s must be 2-D, got shape %s" % (name, tuple(t.shape)))
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("%s must be row-major with unit column stride" % name)
    ld = t.stride(0) if t.shape[0] > 1 else max(t.shape[1], t.stride(0))
    return t.data_ptr(), ld


def det_moe_route(logits, top_k, *, score="softmax", bias=None, n_groups=1, top_groups=1, group_best=2,
                  renormalize=True, scale=1.0, stream=None):
    """The top_k experts of every token and their weights.

    logits [T, E] FP32 or BF16; bias [E] FP32 is added to the scores for the
    choice only. With n_groups > 1 only experts of the best top_groups groups
    are taken, a group's value being the sum of its best group_best choices.
    Returns weights [T, top_k] FP32 and ids [T, top_k] int32, best first, ties
    to the lower index. Experts with a logit of -inf or NaN are masked; a
    choice left over has id -1 and weight 0."""
    p, ld = _logits(logits)
    T, E = logits.shape
    b = None if bias is None else _flat(bias, "bias", _F32, (E,))
    with _on(stream):
        weights = torch.empty((T, top_k), dtype=_F32, device=logits.device)
        ids = torch.empty((T, top_k), dtype=_I32, device=logits.device)
    _run("det_moe_route", p, int(logits.dtype == _F32), b, weights.data_ptr(), ids.data_ptr(), T, E, ld, top_k,
         _score(score), n_groups, top_groups, group_best, int(bool(renormalize)), float(scale),
         _dg._stream_handle(stream))
    return weights, ids


def det_moe_route_bwd(dweights, logits, ids, *, score="softmax", renormalize=True, scale=1.0, stream=None):
    """dlogits [T, E] (the logits' type) from dweights [T, top_k] FP32."""
    p, ld = _logits(logits)
    T, E = logits.shape
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError("ids must be a 2-D tensor")
    k = ids.shape[1]
    i = _flat(ids, "ids", _I32, (T, k))
    d = _flat(dweights, "dweights", _F32, (T, k))
    with _on(stream):
        out = torch.empty((T, E), dtype=logits.dtype, device=logits.device)
    _run("det_moe_route_bwd", d, p, int(logits.dtype == _F32), i, out.data_ptr(), T, E, ld, E, k, _score(score),
         int(bool(renormalize)), float(scale), _dg._stream_handle(stream))
    return out


def det_moe_dispatch(ids, num_experts, *, stream=None):
    """Rows of the experts: ids [T, k] int32 -> offsets [E + 1], rows [T * k]
    (the pair t * k + j of each row, -1 past offsets[E]) and slots [T, k] (the
    row of each pair, -1 for an id outside [0, E)), all int32 on the device."""
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError("ids must be a 2-D tensor")
    T, k = ids.shape
    p = _flat(ids, "ids", _I32, (T, k))
    with _on(stream):
        offsets = torch.empty(num_experts + 1 if num_experts >= 0 else 0, dtype=_I32, device=ids.device)
        rows = torch.empty(T * k, dtype=_I32, device=ids.device)
        slots = torch.empty((T, k), dtype=_I32, device=ids.device)
    _run("det_moe_dispatch", p, offsets.data_ptr(), rows.data_ptr(), slots.data_ptr(), T, num_experts, k,
         _dg._stream_handle(stream))
    return offsets, rows, slots


def _index(t, name, dim):
    if not isinstance(t, torch.Tensor) or t.dim() != dim:
        raise ValueError("%s must be a %d-D tensor" % (name, dim))
    return _flat(t, name, _I32, t.shape)


def det_moe_gather(x, rows, top_k, *, out=None, stream=None):
    """xs[r] = x[rows[r] // top_k] (zero where rows[r] < 0), BF16. Its
    gradient is det_moe_combine(dxs, slots)."""
    p, ld = _mat(x, "x", _BF16)
    T, H = x.shape
    r = _index(rows, "rows", 1)
    R = rows.shape[0]
    with _on(stream):
        out = _new(R, H, _BF16, x.device) if out is None else _given(out, (R, H))
    o, ldo = _mat(out, "out", _BF16)
    _run("det_moe_gather", p, r, o, T, R, H, top_k, ld, ldo, _dg._stream_handle(stream))
    return out


def det_moe_combine(ys, slots, weights=None, *, out=None, stream=None):
    """y[t] = sum over j of weights[t, j] * ys[slots[t, j]] (weights None: 1),
    in FP32 in ascending j, rounded once to BF16."""
    p, ld = _mat(ys, "ys", _BF16)
    R, H = ys.shape
    s = _index(slots, "slots", 2)
    T, k = slots.shape
    w = None if weights is None else _flat(weights, "weights", _F32, (T, k))
    with _on(stream):
        out = _new(T, H, _BF16, ys.device) if out is None else _given(out, (T, H))
    o, ldo = _mat(out, "out", _BF16)
    _run("det_moe_combine", p, s, w, o, T, R, H, k, ld, ldo, _dg._stream_handle(stream))
    return out


def det_moe_combine_bwd(dy, ys, rows, slots, weights, *, stream=None):
    """Gradients of det_moe_combine: dys [T * k, H] BF16 and dweights [T, k] FP32."""
    g, ldg = _mat(dy, "dy", _BF16)
    T, H = dy.shape
    s = _index(slots, "slots", 2)
    k = slots.shape[1]
    if slots.shape[0] != T:
        raise ValueError("dy and slots disagree on the tokens: %d vs %d" % (T, slots.shape[0]))
    r = _flat(rows, "rows", _I32, (T * k,))
    w = _flat(weights, "weights", _F32, (T, k))
    y, ldy = _mat(ys, "ys", _BF16)
    if tuple(ys.shape) != (T * k, H):
        raise ValueError("ys must have shape %s, got %s" % ((T * k, H), tuple(ys.shape)))
    with _on(stream):
        dys = _new(T * k, H, _BF16, dy.device)
        dw = torch.empty((T, k), dtype=_F32, device=dy.device)
    d, ldd = _mat(dys, "dys", _BF16)
    _run("det_moe_combine_bwd", g, y, r, s, w, d, dw.data_ptr(), T, H, k, ldg, ldy, ldd, _dg._stream_handle(stream))
    return dys, dw


def det_fp8_quantize_rows(x, rows=None, top_k=1, *, stream=None):
    """x [T, K] BF16 -> e4m3 [M, K] and one FP32 scale for each row and block
    of 128 columns, a [M, ceil(K / 128)] view of block-major storage. With rows
    (det_moe_dispatch's) row r is x[rows[r] // top_k]: gather and quantise."""
    p, ld = _mat(x, "x", _BF16)
    T, K = x.shape
    r = None if rows is None else _index(rows, "rows", 1)
    M = T if rows is None else rows.shape[0]
    with _on(stream):
        q = _new(M, K, _E4M3, x.device)
        s = torch.empty(((K + BLOCK - 1) // BLOCK, M), dtype=_F32, device=x.device)
    _run("det_fp8_quantize_rows", p, r, q.data_ptr(), s.data_ptr(), T, M, K, top_k, ld, max(q.stride(0), 16), max(M, 1),
         _dg._stream_handle(stream))
    return q, s.t()


def _blocks_for(M, offsets):
    return (M + BLOCK - 1) // BLOCK + (0 if offsets is None else offsets.shape[0] - 1)


def det_fp8_quantize_cols(x, offsets=None, *, stream=None):
    """x [M, K] BF16 -> its transpose in e4m3, [K, blocks * 128], and one FP32
    scale for each column of x and block of 128 rows, [blocks, K]. With offsets
    [G + 1] each group's rows form blocks of their own."""
    p, ld = _mat(x, "x", _BF16)
    M, K = x.shape
    o = None if offsets is None else _index(offsets, "offsets", 1)
    nb = _blocks_for(M, offsets)
    with _on(stream):
        q = torch.empty((K, nb * BLOCK), dtype=_E4M3, device=x.device)
        s = _new(nb, K, _F32, x.device)
    _run("det_fp8_quantize_cols", p, o, q.data_ptr(), s.data_ptr(), M, K, 0 if offsets is None else offsets.shape[0] - 1,
         nb, ld, nb * BLOCK, max(s.stride(0), 4), _dg._stream_handle(stream))
    return q, s


def det_fp8_quantize_tiles(w, transposed=False, *, stream=None):
    """A weight [N, K] (or a stack [G, N, K]) BF16 -> e4m3 of its shape and one
    FP32 scale for each 128 x 128 tile. transposed: the quantised transpose
    [.., K, N] and its scales instead (the input gradient's operand)."""
    if not isinstance(w, torch.Tensor) or w.dim() not in (2, 3):
        raise ValueError("w must be a 2-D or 3-D tensor")
    flat = w.dim() == 2
    p, G, N, K, ld, gap = _mats(w[None] if flat else w, "w", _BF16)
    rt, ct = (N + BLOCK - 1) // BLOCK, (K + BLOCK - 1) // BLOCK
    with _on(stream):
        q = _new(*((K, N) if transposed else (N, K)), _E4M3, w.device, G)
        s = torch.empty((G, ct, rt) if transposed else (G, rt, ct), dtype=_F32, device=w.device)
    a = (q.data_ptr(), s.data_ptr())
    args = (None, None) + a if transposed else a + (None, None)
    ldq, gq = max(q.stride(1), 16), max(q.stride(0), 16)
    _run("det_fp8_quantize_tiles", p, *args, G, N, K, ld, gap, ldq, gq, ldq, gq, _dg._stream_handle(stream))
    return (q[0], s[0]) if flat else (q, s)


def _out_type(out_dtype):
    if out_dtype not in (_BF16, _F32):
        raise TypeError("out_dtype must be torch.bfloat16 or torch.float32, got %s" % (out_dtype,))
    return int(out_dtype == _F32)


def _row_scales(t, name, rows, blocks):
    if not isinstance(t, torch.Tensor) or t.dtype != _F32 or not t.is_cuda:
        raise TypeError("%s must be a float32 CUDA tensor" % name)
    if tuple(t.shape) != (rows, blocks):
        raise ValueError("%s must have shape %s, got %s" % (name, (rows, blocks), tuple(t.shape)))
    return t.data_ptr(), t.stride(0), t.stride(1)


def _tile_scales(t, name, G, rows, cols):
    if not isinstance(t, torch.Tensor) or t.dtype != _F32 or not t.is_cuda:
        raise TypeError("%s must be a float32 CUDA tensor" % name)
    if tuple(t.shape) != (G, rows, cols):
        raise ValueError("%s must have shape %s, got %s" % (name, (G, rows, cols), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _nblk(n):
    return (n + BLOCK - 1) // BLOCK


def det_fp8_gemm(A, a_scale, W, w_scale, *, out_dtype=_BF16, out=None, stream=None):
    """C[M, N] = dequantised A[M, K] @ dequantised W[N, K]^T. A and a_scale
    from det_fp8_quantize_rows, W and w_scale from det_fp8_quantize_tiles. The
    input gradient is det_fp8_gemm(dY, ..) with the transposed weight."""
    a, lda = _mat(A, "A", _E4M3)
    M, K = A.shape
    w, ldw = _mat(W, "W", _E4M3)
    N, K2 = W.shape
    if K2 != K:
        raise ValueError("inner dimensions differ: %d vs %d" % (K, K2))
    sa, sr, sb = _row_scales(a_scale, "a_scale", M, _nblk(K))
    ws = _tile_scales(w_scale[None] if isinstance(w_scale, torch.Tensor) else w_scale, "w_scale", 1, _nblk(N), _nblk(K))
    if out is not None:
        out_dtype = out.dtype
    f32 = _out_type(out_dtype)
    with _on(stream):
        C = _new(M, N, out_dtype, A.device) if out is None else _given(out, (M, N))
    c, ldc = _mat(C, "out", out_dtype)
    _run("det_fp8_gemm", a, sa, w, ws, c, f32, M, N, K, lda, sr, sb, ldw, _nblk(K), ldc, _dg._stream_handle(stream))
    return C


def det_fp8_gemm_grouped(A, a_scale, W, w_scale, offsets, *, out_dtype=_BF16, out=None, stream=None):
    """Rows [offsets[g], offsets[g+1]) of A [M, K] with expert g's weight of W
    [G, N, K] -> C [M, N]. offsets [G + 1] int32 stays on the device; rows
    outside every group become zero."""
    a, lda = _mat(A, "A", _E4M3)
    M, K = A.shape
    w, G, N, K2, ldw, gw = _mats(W, "W", _E4M3)
    if K2 != K:
        raise ValueError("inner dimensions differ: %d vs %d" % (K, K2))
    off = _flat(offsets, "offsets", _I32, (G + 1,))
    sa, sr, sb = _row_scales(a_scale, "a_scale", M, _nblk(K))
    ws = _tile_scales(w_scale, "w_scale", G, _nblk(N), _nblk(K))
    if out is not None:
        out_dtype = out.dtype
    f32 = _out_type(out_dtype)
    with _on(stream):
        C = _new(M, N, out_dtype, A.device) if out is None else _given(out, (M, N))
    c, ldc = _mat(C, "out", out_dtype)
    _run("det_fp8_gemm_grouped", a, sa, w, ws, off, c, f32, G, M, N, K, lda, sr, sb, ldw, gw, _nblk(K),
         _nblk(N) * _nblk(K), ldc, _dg._stream_handle(stream))
    return C


def det_fp8_gemm_wgrad(Yt, y_scale, Xt, x_scale, offsets=None, *, out_dtype=_F32, out=None, stream=None):
    """dW[N, K] = dY^T X from det_fp8_quantize_cols of dY and of X (with the
    same offsets). With offsets [G + 1]: dW [G, N, K], one matrix an expert."""
    y, ldy = _mat(Yt, "Yt", _E4M3)
    N, L = Yt.shape
    x, ldx = _mat(Xt, "Xt", _E4M3)
    K, L2 = Xt.shape
    if L2 != L or L % BLOCK:
        raise ValueError("Yt and Xt must have the same whole number of blocks: %d vs %d columns" % (L, L2))
    nb = L // BLOCK
    sy, ldsy = _mat(y_scale, "y_scale", _F32)
    sx, ldsx = _mat(x_scale, "x_scale", _F32)
    if tuple(y_scale.shape) != (nb, N) or tuple(x_scale.shape) != (nb, K):
        raise ValueError("y_scale and x_scale must have shapes %s and %s, got %s and %s"
                         % ((nb, N), (nb, K), tuple(y_scale.shape), tuple(x_scale.shape)))
    G = 1
    off = None
    M = L
    if offsets is not None:
        off = _index(offsets, "offsets", 1)
        G = offsets.shape[0] - 1
        M = (nb - G) * BLOCK                          # at least the tokens' number
        if G < 0 or M < 0:
            raise ValueError("offsets does not match the blocks of Yt and Xt")
    shape = (N, K) if offsets is None else (G, N, K)
    if out is not None:
        out_dtype = out.dtype
    f32 = _out_type(out_dtype)
    with _on(stream):
        dW = _new(N, K, out_dtype, Yt.device, None if offsets is None else G) if out is None else _given(out, shape)
    d, _, _, _, ldd, gd = _mats(dW[None] if offsets is None else dW, "out", out_dtype)
    _run("det_fp8_gemm_wgrad", y, sy, x, sx, off, d, f32, G, M, N, K, nb, max(ldy, 16), max(ldsy, 4), max(ldx, 16), max(ldsx, 4), ldd, gd,
         _dg._stream_handle(stream))
    return dW


def _tokens(t):
    if not isinstance(t, torch.Tensor) or t.dtype not in (torch.int64, _I32):
        raise TypeError("tokens must be an int64 or int32 tensor")
    if t.dim() != 1:
        raise ValueError("tokens must be 1-D, got shape %s" % (tuple(t.shape),))
    return _flat(t, "tokens", t.dtype, t.shape), int(t.dtype == torch.int64)


def det_embedding(tokens, table, scale=1.0, *, out=None, stream=None):
    """out[t] = scale * table[tokens[t]], rounded once to BF16. A token outside
    the table gives a zero row and an error from det_gemm_check."""
    t, is64 = _tokens(tokens)
    w, ld = _mat(table, "table", _BF16)
    V, H = table.shape
    T = tokens.shape[0]
    with _on(stream):
        out = _new(T, H, _BF16, table.device) if out is None else _given(out, (T, H))
    o, ldo = _mat(out, "out", _BF16)
    _run("det_embedding", t, is64, w, o, T, V, H, float(scale), ld, ldo, _dg._stream_handle(stream))
    return out


def det_embedding_grad(dy, tokens, vocab, scale=1.0, *, padding_idx=None, out_dtype=_F32, out=None, accumulate=False,
                       stream=None):
    """dtable[v] = scale * sum of dy[t] over tokens[t] == v, in a fixed order.
    With accumulate it is added to `out`; rows that never occur are then left
    alone, and become zero otherwise. padding_idx gets no gradient."""
    t, is64 = _tokens(tokens)
    g, ldg = _mat(dy, "dy", _BF16)
    T, H = dy.shape
    if tokens.shape[0] != T:
        raise ValueError("dy and tokens disagree on the tokens: %d vs %d" % (T, tokens.shape[0]))
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    if padding_idx is not None and not 0 <= padding_idx < vocab:
        raise ValueError("padding_idx must be in [0, vocab)")
    if out is not None:
        out_dtype = out.dtype
    f32 = _out_type(out_dtype)
    size = _fn("det_embedding_grad_workspace")(T, vocab, H)
    with _on(stream):
        out = _new(vocab, H, out_dtype, dy.device) if out is None else _given(out, (vocab, H))
        ws = torch.empty(max(size, 256), dtype=torch.uint8, device=dy.device)
    o, ldo = _mat(out, "out", out_dtype)
    _run("det_embedding_grad", g, t, is64, o, f32, T, vocab, H, float(scale), -1 if padding_idx is None else padding_idx,
         int(bool(accumulate)), ldg, ldo, ws.data_ptr(), ws.numel(), _dg._stream_handle(stream))
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
