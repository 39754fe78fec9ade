"""Attention operators (include/det_attn.h) for PyTorch tensors.

Argument marshalling only, as in _ops.py. Heads are [tokens, heads, D] BF16
tensors, views of one projection's output among them (unit stride in D, the
other strides multiples of 16 bytes); D is a multiple of 8, at most 128. A
paged cache is [pages, page_size, heads, D], in any order of strides but D's.

  det_rope(x, cos, sin, positions)                      -> y       (gradient: inverse=True)
  det_kv_append(q, k, v, cos, sin, positions, slots, k_cache, v_cache) -> rotated q
  det_attn_decode(q, k_cache, v_cache, table, lengths)  -> out
  det_attn(q, k, v, bounds=None, k_bounds=None)         -> out, lse
  det_attn_bwd(dout, q, k, v, out, lse, bounds=None, k_bounds=None) -> dq, dk, dv
"""
from __future__ import annotations

from . import _ops
from ._ops import _on


def det_rope(x, cos, sin, positions, *, interleaved=False, inverse=False, out=None, stream=None):
    """x [T, H, D] with the first 2 * cos.shape[1] columns of every head turned
    by its token's angle. cos and sin [P, rot / 2] FP32, positions [T] int32
    rows of them. Pairs are columns (i, i + rot / 2), or (2i, 2i + 1) with
    interleaved. inverse turns back: the gradient. out may be x itself. A
    position outside the tables gives a zero row and an error from
    det_gemm_check."""
    return _on(stream, _ops._native.rope, x, cos, sin, positions, interleaved, inverse, out)


def det_kv_append(q, k, v, cos, sin, positions, slots, k_cache, v_cache, *, interleaved=False, out=None, stream=None):
    """Turns k [T, KV, D] as det_rope does and stores it and v in the caches:
    token t in row slots[t] (int32; page * page_size + place, -1: nowhere).
    Slots other than -1 must be distinct. Returns q [T, H, D] turned (None for
    q None)."""
    return _on(stream, _ops._native.kv_append, q, k, v, cos, sin, positions, slots, k_cache, v_cache, interleaved, out)


def det_attn_decode(q, k_cache, v_cache, table, lengths, *, scale=None, window=None, sinks=0, out=None, stream=None):
    """Attention of one new token a sequence: q [B, H, D] over the first
    lengths[b] tokens of the pages table[b] (int32 [B, max_pages]), the new
    token's own key among them. With a window only the last `window` keys and
    the first `sinks` are seen. scale: 1 / sqrt(D) unless given. A sequence of
    length 0 gives zeros. The same in any batch; det_attn's row of the same
    token differs by roundings."""
    return _on(stream, _ops._native.attn_decode, q, k_cache, v_cache, table, lengths, scale, window, sinks, out)


def det_attn(q, k, v, bounds=None, k_bounds=None, *, scale=None, window=None, sinks=0, out=None, stream=None):
    """Causal attention of packed sequences: q [T, H, D], k and v [S, KV, D];
    sequence n has the queries bounds[n]:bounds[n + 1] and the keys
    k_bounds[n]:k_bounds[n + 1] (int32 on the device; None: the queries'), its
    last query at its last key. bounds None: one sequence. With a window a
    query sees the last `window` keys up to its own and the first `sinks`.
    Returns out [T, H, D] and lse [H, T] FP32."""
    return _on(stream, _ops._native.attn, q, k, v, bounds, k_bounds, scale, window, sinks, out)


def det_attn_bwd(dout, q, k, v, out, lse, bounds=None, k_bounds=None, *, scale=None, window=None, sinks=0, stream=None):
    """Gradients dq, dk, dv of det_attn, from its inputs and results. out and lse
    may be those of more keys than k and v (results over several ranges of
    keys, joined): the gradients are then this range's part."""
    return _on(stream, _ops._native.attn_bwd, dout, q, k, v, out, lse, bounds, k_bounds, scale, window, sinks)


__all__ = ["det_rope", "det_kv_append", "det_attn_decode", "det_attn", "det_attn_bwd"]
