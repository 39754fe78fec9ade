"""Mixture-of-experts operators (include/det_ops.h) for PyTorch tensors.

Argument marshalling only, in the manner of the det_gemm binding: every
function takes CUDA tensors of the current device (of `stream`'s, where one is
given), checks their types and layouts, allocates what is not given with
PyTorch (on the stream the work runs on) and calls the C function of the same
name. The marshalling itself is native code
(binding/ops_native.cpp), because a decode-sized call is bound by it. There is
no fallback.

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

import torch

import invariant_deterministic_gemm_gb300 as _dg

_BF16, _F32 = torch.bfloat16, torch.float32
_SCORES = {"softmax": 0, "sigmoid": 1}
_OUT_TYPES = {_BF16: 0, _F32: 1}

_native = None


class _Unloaded:
    """Stands in for the native module until the first call (importing the
    package needs no built library)."""

    def __getattr__(self, name):
        global _native
        _dg.lib()                                     # raises if nothing was built
        try:
            from . import _ops_native
        except ImportError as e:
            raise ImportError("the operators' native binding is not built or does not load (%s); _build.build() needs a C++ "
                              "compiler and PyTorch's and Python's headers for it" % e) from e
        _native = _ops_native
        return getattr(_native, name)


_native = _Unloaded()


def _score(score):
    s = _SCORES.get(score)
    if s is None:
        raise ValueError("score must be 'softmax' or 'sigmoid', got %r" % (score,))
    return s


def _fp32(out_dtype):
    f = _OUT_TYPES.get(out_dtype)
    if f is None:
        raise TypeError("out_dtype must be torch.bfloat16 or torch.float32, got %s" % (out_dtype,))
    return f


def _on(stream, fn, *args):
    """fn(*args) with its work and its allocations on the given stream: a
    torch.cuda.Stream, or any object whose cuda_stream is a stream's handle."""
    if stream is None:
        return fn(*args)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream.cuda_stream))
    with torch.cuda.stream(stream):
        return fn(*args)


def det_moe_route(logits, top_k, *, score="softmax", bias=None, n_groups=1, top_groups=1, group_best=2,
                  renormalize=True, scale=1.0, stream=None):
    """The top_k experts of every token and their weights.

    logits [T, E] FP32 or BF16; bias [E] FP32 is added to the scores for the
    choice only. With n_groups > 1 only experts of the best top_groups groups
    are taken, a group's value being the sum of its best group_best choices.
    Returns weights [T, top_k] FP32 and ids [T, top_k] int32, best first, ties
    to the lower index. Experts with a logit (or bias) of -inf or NaN are
    masked; a choice left over has id -1 and weight 0. A logit of +inf is
    chosen like the largest finite FP32 value, and makes its row's softmax
    weights NaN; a bias of +inf puts its expert first."""
    return _on(stream, _native.route, logits, top_k, _score(score), bias, n_groups, top_groups, group_best, renormalize, scale)


def det_moe_route_bwd(dweights, logits, ids, *, score="softmax", renormalize=True, scale=1.0, stream=None):
    """dlogits [T, E] (the logits' type) from dweights [T, top_k] FP32."""
    return _on(stream, _native.route_bwd, dweights, logits, ids, _score(score), renormalize, scale)


def det_moe_dispatch(ids, num_experts, *, stream=None):
    """Rows of the experts: ids [T, k] int32 -> offsets [E + 1], rows [T * k]
    (the pair t * k + j of each row, -1 past offsets[E]) and slots [T, k] (the
    row of each pair, -1 for an id outside [0, E)), all int32 on the device."""
    return _on(stream, _native.dispatch, ids, num_experts)


def det_moe_gather(x, rows, top_k, *, out=None, stream=None):
    """xs[r] = x[rows[r] // top_k] (zero where rows[r] < 0), BF16. Its
    gradient is det_moe_combine(dxs, slots)."""
    return _on(stream, _native.gather, x, rows, top_k, out)


def det_moe_combine(ys, slots, weights=None, *, out=None, stream=None):
    """y[t] = sum over j of weights[t, j] * ys[slots[t, j]] (weights None: 1),
    in FP32 in ascending j, rounded once to BF16."""
    return _on(stream, _native.combine, ys, slots, weights, out)


def det_moe_combine_bwd(dy, ys, rows, slots, weights, *, stream=None):
    """Gradients of det_moe_combine: dys [T * k, H] BF16 and dweights [T, k] FP32."""
    return _on(stream, _native.combine_bwd, dy, ys, rows, slots, weights)


def det_fp8_quantize_rows(x, rows=None, top_k=1, *, stream=None):
    """x [T, K] BF16 -> e4m3 [M, K] and one FP32 scale for each row and block
    of 128 columns, a [M, ceil(K / 128)] tensor stored block by block. With
    rows (det_moe_dispatch's) row r is x[rows[r] // top_k]: gather and
    quantise."""
    return _on(stream, _native.quantize_rows, x, rows, top_k)


def det_fp8_quantize_cols(x, offsets=None, *, stream=None):
    """x [M, K] BF16 -> its transpose in e4m3, [K, blocks * 128], and one FP32
    scale for each column of x and block of 128 rows, [blocks, K]. With offsets
    [G + 1] each group's rows form blocks of their own."""
    return _on(stream, _native.quantize_cols, x, offsets)


def det_fp8_quantize_tiles(w, transposed=False, *, stream=None):
    """A weight [N, K] (or a stack [G, N, K]) BF16 -> e4m3 of its shape and one
    FP32 scale for each 128 x 128 tile. transposed: the quantised transpose
    [.., K, N] and its scales instead (the input gradient's operand)."""
    return _on(stream, _native.quantize_tiles, w, transposed)


def det_fp8_gemm(A, a_scale, W, w_scale, *, out_dtype=_BF16, out=None, stream=None):
    """C[M, N] = dequantised A[M, K] @ dequantised W[N, K]^T. A and a_scale
    from det_fp8_quantize_rows, W and w_scale from det_fp8_quantize_tiles. The
    input gradient is det_fp8_gemm(dY, ..) with the transposed weight."""
    return _on(stream, _native.gemm, A, a_scale, W, w_scale, _fp32(out_dtype), out)


def det_fp8_gemm_grouped(A, a_scale, W, w_scale, offsets, *, out_dtype=_BF16, out=None, stream=None):
    """Rows [offsets[g], offsets[g+1]) of A [M, K] with expert g's weight of W
    [G, N, K] -> C [M, N]. offsets [G + 1] int32 stays on the device; rows
    outside every group become zero."""
    return _on(stream, _native.gemm_grouped, A, a_scale, W, w_scale, offsets, _fp32(out_dtype), out)


def det_fp8_gemm_wgrad(Yt, y_scale, Xt, x_scale, offsets=None, *, out_dtype=_F32, out=None, stream=None):
    """dW[N, K] = dY^T X from det_fp8_quantize_cols of dY and of X (with the
    same offsets). With offsets [G + 1]: dW [G, N, K], one matrix an expert."""
    return _on(stream, _native.gemm_wgrad, Yt, y_scale, Xt, x_scale, offsets, _fp32(out_dtype), out)


def det_embedding(tokens, table, scale=1.0, *, out=None, stream=None):
    """out[t] = scale * table[tokens[t]], rounded once to BF16. A token outside
    the table gives a zero row and an error from det_gemm_check."""
    return _on(stream, _native.embedding, tokens, table, scale, out)


def det_embedding_grad(dy, tokens, vocab, scale=1.0, *, padding_idx=None, out_dtype=_F32, out=None, accumulate=False,
                       stream=None):
    """dtable[v] = scale * sum of dy[t] over tokens[t] == v, in a fixed order.
    With accumulate it is added to `out`; rows that never occur are then left
    alone, and become zero otherwise. padding_idx gets no gradient."""
    return _on(stream, _native.embedding_grad, dy, tokens, vocab, scale, padding_idx, _fp32(out_dtype), out, accumulate)


def det_ops_check(stream=None) -> int:
    """Synchronise the stream and return (and clear) these operators' device status."""
    return int(_dg.lib().det_ops_check(_dg._stream_handle(stream)))


def det_ops_debug_force_timeout(enable: bool) -> None:
    """Test hook: make every later 8-bit product time out on purpose (see det_ops.h)."""
    _native.force_timeout(enable)


__all__ = [
    "det_moe_route", "det_moe_route_bwd", "det_moe_dispatch", "det_moe_gather", "det_moe_combine",
    "det_moe_combine_bwd", "det_fp8_quantize_rows", "det_fp8_quantize_cols", "det_fp8_quantize_tiles",
    "det_fp8_gemm", "det_fp8_gemm_grouped", "det_fp8_gemm_wgrad", "det_embedding", "det_embedding_grad",
    "det_ops_check", "det_ops_debug_force_timeout",
]
