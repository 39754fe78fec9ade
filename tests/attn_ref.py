"""The attention operators in 64 bits, and how far BF16 results may be off.

A kernel rounds P (and dS) once to BF16 for its second product, relative 2^-8,
and its result once; the rest is FP32. The bounds below add those two to the
FP32 errors of a score (its products' sum, the argument of the exponential)."""
import math

import torch

F64 = torch.float64
U16, U32 = 2.0 ** -8, 2.0 ** -24        # half a step, relative: BF16, FP32


def f64(t):
    return t.detach().to("cpu", F64)


def spans(bounds, n):
    if bounds is None:
        return [(0, n)]
    b = [int(x) for x in bounds]
    return list(zip(b[:-1], b[1:]))


def visible(nq, nk, window=None, sinks=0):
    i = torch.arange(nq)[:, None] + nk - nq
    j = torch.arange(nk)[None]
    vis = j <= i
    if window is not None:
        vis = vis & ((i - j < window) | (j < sinks))
    return vis


def scores(q, k, vis, scale):
    """Masked scores, and what FP32 may make of one: its sum's error and the exponential's argument's."""
    s = q @ k.T * scale
    off = (q.abs() @ k.abs().T) * scale * (q.shape[1] + 4) * U32
    s, off = s.masked_fill(~vis, -math.inf), off.masked_fill(~vis, 0.0)
    return s, off


def one(q, k, v, vis, scale):
    """out, lse and their bounds for one head."""
    v = torch.where(vis.any(0)[:, None], v, torch.zeros((), dtype=F64))        # what nobody sees may be anything
    k = torch.where(vis.any(0)[:, None], k, torch.zeros((), dtype=F64))
    s, off = scores(q, k, vis, scale)
    lse = torch.logsumexp(s, 1)
    some = vis.any(1)
    p = torch.where(vis, torch.exp(s - torch.where(some, lse, torch.zeros_like(lse))[:, None]), torch.zeros((), dtype=F64))
    out, size = p @ v, p @ v.abs()
    # exponent: the score's error and the rounding of score and maximum, both at most the largest score
    arg = (off.amax(1) + 4 * U32 * s.masked_fill(~vis, 0.0).abs().amax(1)) if vis.shape[1] else torch.zeros(len(q), dtype=F64)
    rel = 2 * arg + (vis.shape[1] + 16) * U32 * 4
    tol = U16 * (size + out.abs()) * 1.01 + size * rel[:, None] + 1e-30
    return out, lse, tol, arg + 64 * U32 * (1 + torch.where(some, lse, torch.zeros_like(lse)).abs()), p


def attention(q, k, v, bounds=None, k_bounds=None, scale=None, window=None, sinks=0):
    """out, lse, and the bounds of both."""
    q, k, v = f64(q), f64(k), f64(v)
    T, H, D = q.shape
    KV = k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    out, tol = torch.zeros_like(q), torch.full_like(q, 1e-30)
    lse, ltol = torch.full((H, T), -math.inf, dtype=F64), torch.zeros((H, T), dtype=F64)
    for (a, b), (c, d) in zip(spans(bounds, T), spans(bounds if k_bounds is None else k_bounds, len(k))):
        vis = visible(b - a, d - c, window, sinks)
        for h in range(H):
            g = h // (H // KV)
            out[a:b, h], lse[h, a:b], tol[a:b, h], ltol[h, a:b], _ = one(q[a:b, h], k[c:d, g], v[c:d, g], vis, scale)
    return out, lse, tol, ltol


def gradients(dout, q, k, v, out, lse, bounds=None, k_bounds=None, scale=None, window=None, sinks=0):
    """dq, dk, dv from the inputs as they are (out and lse among them), and their bounds."""
    dout, q, k, v, out, lse = (f64(x) for x in (dout, q, k, v, out, lse))
    T, H, D = q.shape
    KV = k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    tq, tk, tv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for (a, b), (c, d) in zip(spans(bounds, T), spans(bounds if k_bounds is None else k_bounds, len(k))):
        vis = visible(b - a, d - c, window, sinks)
        if not vis.any():
            continue
        for h in range(H):
            g = h // (H // KV)
            qh, kh, vh, do, o = q[a:b, h], k[c:d, g], v[c:d, g], dout[a:b, h], out[a:b, h]
            s, off = scores(qh, kh, vis, scale)
            L = torch.where(vis.any(1), lse[h, a:b], torch.zeros(b - a, dtype=F64))[:, None]
            p = torch.where(vis, torch.exp(s - L), torch.zeros((), dtype=F64))
            rel = 2 * off + 8 * U32 * (s.masked_fill(~vis, 0.0).abs() + L.abs() + 2)        # of an element of P
            dp, delta = do @ vh.T, (do * o).sum(1, keepdim=True)
            ds = p * (dp - delta)
            dp_off = (do.abs() @ vh.abs().T + (do.abs() * o.abs()).sum(1, keepdim=True)) * (D + 8) * U32
            ds_off = ds.abs() * (U16 * 1.01 + 2 * rel) + p * dp_off * 1.01
            p_off = p * (U16 * 1.01 + 2 * rel)
            n = (vis.shape[0] * (H // KV) + vis.shape[1] + 16) * U32
            dq[a:b, h] = scale * ds @ kh
            tq[a:b, h] = scale * (ds_off + ds.abs() * n) @ kh.abs()
            dk[c:d, g] += scale * ds.T @ qh
            tk[c:d, g] += scale * (ds_off + ds.abs() * n).T @ qh.abs()
            dv[c:d, g] += p.T @ do
            tv[c:d, g] += (p_off + p * n).T @ do.abs()
    return [(x, t + U16 * 1.01 * x.abs() + 1e-30) for x, t in ((dq, tq), (dk, tk), (dv, tv))]


def turned(x, cos, sin, pos, interleaved=False, inverse=False):
    """det_rope in 64 bits and its bound: the two products' and their sum's roundings, and the result's."""
    x, c, s = f64(x), f64(cos)[pos.cpu().long()][:, None], f64(sin)[pos.cpu().long()][:, None]
    if inverse:
        s = -s
    half = c.shape[2]
    y, tol = x.clone(), torch.zeros_like(x)
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    tol[..., a] = 2 * U32 * ((x[..., a] * c).abs() + (x[..., b] * s).abs())
    tol[..., b] = 2 * U32 * ((x[..., b] * c).abs() + (x[..., a] * s).abs())
    return y, torch.where(tol > 0, tol + U16 * 1.01 * y.abs(), tol)


def assert_within(got, want, tol, what=""):
    got = f64(got)
    assert got.shape == want.shape, what
    bad = ~((got - want).abs() <= tol) & ~(got == want)
    assert not bad.any(), "%s: %d of %d off, the first at %s: %r, wanted %r within %r" % (
        what, int(bad.sum()), bad.numel(), tuple(bad.nonzero()[0].tolist()), float(got[bad][0]), float(want[bad][0]), float(tol[bad][0]))
