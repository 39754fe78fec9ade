"""Plain 64-bit implementations of the mixture-of-experts operators, written
from their definitions with numpy, for the tests."""
import numpy as np
import torch

BLOCK = 128
EPS_BF16 = torch.finfo(torch.bfloat16).eps / 2      # half a step of a rounding to BF16
EPS_F32 = torch.finfo(torch.float32).eps / 2


def f64(t):
    return t.detach().to("cpu").double().numpy()


def route(logits, k, score="softmax", bias=None, n_groups=1, top_groups=1, group_best=2, renormalize=True, scale=1.0):
    """(weights, ids) by a loop over the rows; logits a float64 array."""
    T, E = logits.shape
    W = np.zeros((T, k))
    ids = np.full((T, k), -1, dtype=np.int64)
    for t in range(T):
        l = logits[t]
        ok = l > -np.inf                             # not -inf, not NaN
        s = np.zeros(E)
        if ok.any():
            if score == "softmax":
                e = np.exp(l[ok] - l[ok].max())
                s[ok] = e / e.sum()
            else:
                s[ok] = 1.0 / (1.0 + np.exp(-l[ok]))
        c = s + bias if bias is not None else s
        if n_groups > 1:
            size = E // n_groups
            val = np.full(n_groups, -np.inf)
            for g in range(n_groups):
                v = sorted((c[e] for e in range(g * size, (g + 1) * size) if ok[e]), reverse=True)[:group_best]
                if v:
                    val[g] = sum(v)
            order = sorted(range(n_groups), key=lambda g: (-val[g], g))[:top_groups]
            for g in range(n_groups):
                if g not in order:
                    ok = ok.copy()
                    ok[g * size:(g + 1) * size] = False
        rank = c if bias is not None else l          # without a bias the logits' order is the scores'
        cand = sorted((e for e in range(E) if ok[e]), key=lambda e: (-rank[e], e))[:k]
        for j, e in enumerate(cand):
            ids[t, j] = e
            W[t, j] = s[e]
        if renormalize and cand:
            W[t] /= W[t].sum() + (1e-20 if score == "sigmoid" else 0.0)
    return W * scale, ids


def weights_of(logits, ids, score, renormalize, scale):
    """The weights as a smooth function of the logits, for fixed ids (float64 torch)."""
    live = logits > -float("inf")
    if score == "softmax":
        s = torch.softmax(torch.where(live, logits, torch.full_like(logits, -float("inf"))), 1)
        s = torch.nan_to_num(s, nan=0.0)
    else:
        s = torch.sigmoid(torch.where(live, logits, torch.zeros_like(logits))) * live
    w = torch.gather(s, 1, ids.clamp(min=0)) * (ids >= 0)
    if renormalize:
        S = w.sum(1, keepdim=True) + (1e-20 if score == "sigmoid" else 0.0)
        w = w / torch.where(S > 0, S, torch.ones_like(S))
    return w * scale


def route_gradient(logits, ids, dw, score, renormalize, scale):
    """d <dw, weights> / d logits by the formula, float64 arrays, ids fixed."""
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        live = logits[t] > -np.inf
        sel = [(int(e), g * scale) for e, g in zip(ids[t], dw[t]) if e >= 0]
        if not sel:
            continue
        s = np.zeros(E)
        if score == "softmax":
            s[live] = np.exp(logits[t][live] - logits[t][live].max())
            s /= s.sum()
        else:
            s[live] = 1.0 / (1.0 + np.exp(-logits[t][live]))
        e, g = np.array([a for a, _ in sel]), np.array([b for _, b in sel])
        if renormalize:
            S = s[e].sum() + (1e-20 if score == "sigmoid" else 0.0)
            g = (g - (s[e] / S * g).sum()) / S       # now the slope with respect to the chosen scores
        if score == "sigmoid":
            out[t, e] = s[e] * (1.0 - s[e]) * g
        elif renormalize:
            out[t, e] = s[e] * g                     # the softmax's own sum cancels
        else:
            d = np.zeros(E)
            d[e] = g
            out[t] = s * (d - (s * d).sum())
    return out


def dispatch(ids, E):
    flat = ids.reshape(-1)
    rows = [i for e in range(E) for i in np.nonzero(flat == e)[0]]
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(E)])])
    slots = np.full(flat.size, -1, dtype=np.int64)
    for r, i in enumerate(rows):
        slots[i] = r
    rows = np.array(rows + [-1] * (flat.size - len(rows)), dtype=np.int64)
    return offsets, rows, slots.reshape(ids.shape)


def e4m3(v):
    """float64 -> nearest e4m3 value, ties to even, at most 448."""
    _, ex = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(ex - 1, -6) - 3)
    return np.clip(np.rint(v / step) * step, -448.0, 448.0)


def quantize(x, axis=1):
    """x (float64 array) in blocks of 128 along `axis` -> (q values, float32 scales)."""
    x = x if axis == 1 else x.T
    n, K = x.shape
    nb = (K + BLOCK - 1) // BLOCK
    q = np.zeros((n, K))
    s = np.zeros((n, nb), dtype=np.float32)
    for b in range(nb):
        v = x[:, b * BLOCK:(b + 1) * BLOCK]
        amax = np.maximum(np.abs(v).max(1), 2.0 ** -100)
        s[:, b] = amax.astype(np.float32) / np.float32(448.0)
        with np.errstate(over="ignore", invalid="ignore"):
            q[:, b * BLOCK:(b + 1) * BLOCK] = e4m3(v * 448.0 / amax[:, None])
    return (q, s) if axis == 1 else (q.T, s.T)


def dequantize(q, s):
    return q * np.repeat(s.astype(np.float64), BLOCK, axis=1)[:, :q.shape[1]]


def quantize_tiles(w):
    N, K = w.shape
    q = np.zeros((N, K))
    s = np.zeros(((N + 127) // 128, (K + 127) // 128), dtype=np.float32)
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            v = w[i * 128:(i + 1) * 128, j * 128:(j + 1) * 128]
            amax = max(np.abs(v).max(), 2.0 ** -100)
            s[i, j] = np.float32(amax) / np.float32(448.0)
            q[i * 128:(i + 1) * 128, j * 128:(j + 1) * 128] = e4m3(v * 448.0 / amax)
    return q, s


def dequantize_tiles(q, s):
    return q * np.repeat(np.repeat(s.astype(np.float64), 128, 0), 128, 1)[:q.shape[0], :q.shape[1]]


def e4m3_tensor(q):
    """float64 e4m3 values -> torch e4m3 tensor with a row pitch of whole 16 bytes (CPU)."""
    n, K = q.shape
    t = torch.zeros((n, max(16, (K + 15) // 16 * 16)), dtype=torch.float32)
    t[:, :K] = torch.from_numpy(np.ascontiguousarray(q)).float()
    return t.to(torch.float8_e4m3fn)


def product_tolerance(absdot, blocks, out_dtype, want):
    """Largest error of a block-scaled product. Inside a block the tensor
    core adds 128 exact products in FP32, each addition off by at most one
    unit in the last place of the sum of magnitudes (2^-23, truncation
    included); across blocks each fused multiply-add and the scales' product
    round once (2^-24 each, one more for the stored scales' own product);
    then one rounding to the output's type."""
    tol = absdot * (128 * 2.0 ** -23 + (blocks + 3) * 2.0 ** -24)
    half = EPS_BF16 if out_dtype == torch.bfloat16 else EPS_F32
    return tol + half * (np.abs(want) + tol) + 1e-38
