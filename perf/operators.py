"""Performance cases of the mixture-of-experts operators.

Each case runs one operator the way a program uses it: routing to experts
(with its gradient), dispatch and combine around the experts' products,
the 8-bit block-scaled product (dense and per expert, with the gradients),
and the embedding lookup with its gradient. ``run`` computes the operator
in elementary torch operations, or, when ``own`` is set, calls the
package's operators; ``exact`` computes it in 64 bits from the definition.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
AMAX_MIN = 2.0 ** -100
SIGMOID_EPS = 1e-20


# ------------------------------------------------------------------ cases

def listed():
    return [
        # Router of a decode step: a handful of tokens, eight experts.
        dict(name="route_decode", op="route", T=17, E=8, k=2, score="softmax", bias=False, groups=1, top_groups=1,
             renorm=True, scale=1.0, dtype="fp32", train=False),
        # Router of a prompt: many experts in groups, a balance bias, sigmoid scores.
        dict(name="route_prefill_groups", op="route", T=8192, E=256, k=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, renorm=True, scale=2.5, dtype="fp32", train=False),
        # Router of a training step, odd sizes, BF16 logits, forward and gradient.
        dict(name="route_train", op="route", T=4099, E=60, k=4, score="softmax", bias=False, groups=1, top_groups=1,
             renorm=False, scale=1.0, dtype="bf16", train=True),
        # Rows to experts and back in a decode step.
        dict(name="experts_decode", op="experts", T=17, E=8, k=2, H=4096, train=False),
        # The same in a training step of 8192 tokens, with all gradients.
        dict(name="experts_train", op="experts", T=8192, E=64, k=6, H=4096, train=True),
        # QKV projection of a decode step on 8-bit weights.
        dict(name="fp8_decode", op="fp8", M=3, N=12288, K=4096, out="bf16", train=False),
        # MLP up-projection of a ragged prompt.
        dict(name="fp8_prefill_ragged", op="fp8", M=1021, N=14336, K=4096, out="bf16", train=False),
        # MLP up-projection of a training step: forward, input and weight gradient.
        dict(name="fp8_train", op="fp8", M=8192, N=14336, K=4096, out="fp32", train=True),
        # The experts' products of a decode step: few rows for each expert.
        dict(name="fp8_experts_decode", op="fp8_experts", M=34, N=1792, K=4096, E=8, out="bf16", train=False),
        # The experts' products of a training step: uneven loads, one expert without rows.
        dict(name="fp8_experts_train", op="fp8_experts", M=16384, N=1792, K=4096, E=8, out="bf16", train=True),
        # A small model's embedding in a training step, odd sizes, FP32 gradient.
        dict(name="embed_small", op="embed", T=333, V=32003, H=1000, scale=31.622776, grad="fp32"),
        # The embedding of a training step on a large vocabulary.
        dict(name="embed_train", op="embed", T=8192, V=151936, H=4096, scale=1.0, grad="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "experts", "fp8", "fp8_experts", "embed"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * rng.randint(max(2, 8 // groups), 256 // groups)
        top_groups = rng.randint(1, groups)
        k = rng.randint(1, min(8, E // groups * top_groups))
        return dict(op=op, T=_log(rng, 1, 8192), E=E, k=k, score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, groups=groups, top_groups=top_groups, renorm=rng.random() < 0.5,
                    scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["fp32", "bf16"]), train=rng.random() < 0.5)
    if op == "experts":
        T = _log(rng, 1, 8192)
        return dict(op=op, T=T, E=_log(rng, 2, 256), k=rng.randint(1, 6), H=_log(rng, 64, 4096),
                    train=rng.random() < 0.5)
    if op == "fp8":
        train = rng.random() < 0.5
        return dict(op=op, M=_log(rng, 1, 8192), N=_log(rng, 64, 14336), K=_log(rng, 64, 4096),
                    out=rng.choice(["bf16", "fp32"]), train=train)
    if op == "fp8_experts":
        return dict(op=op, M=_log(rng, 1, 16384), N=_log(rng, 64, 1792), K=_log(rng, 64, 4096), E=rng.randint(1, 24),
                    out=rng.choice(["bf16", "fp32"]), train=rng.random() < 0.5)
    V = _log(rng, 64, 151936)
    return dict(op=op, T=_log(rng, 1, 8192), V=V, H=_log(rng, 64, 4096), scale=rng.choice([1.0, 45.254834]),
                grad=rng.choice(["bf16", "fp32"]) if V <= 65536 else "bf16")


def work(case):
    c = case
    if c["op"] == "route":
        es = 4 if c["dtype"] == "fp32" else 2
        b = c["T"] * (c["E"] * es + c["k"] * 8) + (4 * c["E"] if c["bias"] else 0)
        f = 12.0 * c["T"] * c["E"]
        if c["train"]:
            b += c["T"] * (c["E"] * es + c["k"] * 4)      # dw in, dlogits out
            f *= 2
        return {"bytes": b, "flops": f}
    if c["op"] == "experts":
        row, T, R = 2 * c["H"], c["T"], c["T"] * c["k"]
        b = 2 * T * row + 2 * R * row + R * 16 + 4 * (c["E"] + 1)   # x, y, xs, ys; ids, weights, rows, slots
        f = 2.0 * R * c["H"]
        if c["train"]:
            b += T * row + 2 * R * row + T * row + R * 4  # dy, dys, dxs; dx, dw
            f += 4.0 * R * c["H"]
        return {"bytes": b, "flops": f}
    if c["op"] in ("fp8", "fp8_experts"):
        M, N, K, E = c["M"], c["N"], c["K"], c.get("E", 1)
        es = 4 if c["out"] == "fp32" else 2
        b = 2 * M * K + E * N * K + 2 * M * N
        f = 2.0 * M * N * K
        if c["train"]:
            b += 2 * M * N + E * N * K + 2 * M * K + es * E * N * K
            f *= 3
        return {"bytes": b, "flops": f}
    T, V, H = c["T"], c["V"], c["H"]
    es = 4 if c["grad"] == "fp32" else 2
    return {"bytes": 4 * T * H + 8 * T + 2 * T * H + es * V * H, "flops": 2.0 * T * H}


# ----------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)


def _padded(rows, cols, dtype, per16):
    """A [rows, cols] tensor whose row pitch is a multiple of 16 bytes."""
    return torch.zeros((rows, (cols + per16 - 1) // per16 * per16), dtype=dtype, device="cuda")[:, :cols]


def _randn(g, rows, cols, std, outliers=False):
    x = torch.randn((rows, cols), generator=g, device="cuda") * std
    if outliers:      # a few channels far larger than the rest, as hidden states have
        ch = torch.rand(cols, generator=g, device="cuda") < 0.005
        x = torch.where(ch[None, :], x * 20.0, x)
    t = _padded(rows, cols, torch.bfloat16, 8)
    t.copy_(x)
    return t


def _blocks(x, dim):
    """x with dimension `dim` padded by zeros to whole blocks and split in (blocks, BLOCK)."""
    n = x.shape[dim]
    nb = (n + BLOCK - 1) // BLOCK
    if nb * BLOCK != n:
        pad = list(x.shape)
        pad[dim] = nb * BLOCK - n
        x = torch.cat([x, x.new_zeros(pad)], dim)
    return x.reshape(x.shape[:dim] + (nb, BLOCK) + x.shape[dim + 1:])


def _quantize_weights(w):
    """[E, N, K] FP32 -> e4m3 values (row pitch a multiple of 16) and one scale for each 128 x 128 tile."""
    N, K = w.shape[1:]
    t = _blocks(_blocks(w, 1), 3)               # [E, nb, 128, kb, 128]
    amax = t.abs().amax((2, 4), keepdim=True).clamp(min=AMAX_MIN)
    q = (t * E4M3_MAX / amax).to(torch.float8_e4m3fn)
    q = q.reshape(t.shape[0], t.shape[1] * BLOCK, -1)[:, :N, :K]
    s = (amax / E4M3_MAX).reshape(t.shape[0], t.shape[1], t.shape[3])
    return _pitch16(q), s.contiguous()


def _pitch16(q):
    E, N, K = q.shape
    out = torch.zeros((E, N, (K + 15) // 16 * 16), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)[:, :, :K]
    out.copy_(q)
    return out


def _counts(g, M, E):
    """Rows of each expert: uneven, one expert without any when there are enough."""
    p = torch.rand(E, generator=g, device="cuda", dtype=torch.float64) ** 2 + 0.05
    if E >= 4:
        p[E // 2] = 0.0
    edges = torch.floor(torch.cumsum(p / p.sum(), 0) * M + 0.5).to(torch.int64)
    edges[-1] = M
    return torch.cat([edges.new_zeros(1), edges])


def prepare(case, seed):
    c, g = case, _gen(seed)
    if c["op"] == "route":
        T, E = c["T"], c["E"]
        dt = torch.float32 if c["dtype"] == "fp32" else torch.bfloat16
        x = torch.randn((T, E), generator=g, device="cuda") * 1.5
        x = x + torch.randn(E, generator=g, device="cuda") * 0.5         # experts differ in popularity
        off = torch.rand((T, E), generator=g, device="cuda") < 0.002     # switched-off experts
        x = torch.where(off, torch.full_like(x, -math.inf), x)
        pad = torch.rand(T, generator=g, device="cuda") < 0.01           # padding tokens: nothing left to choose
        x = torch.where(pad[:, None], torch.full_like(x, -math.inf), x)
        logits = _padded(T, E, dt, 4 if dt == torch.float32 else 8)
        logits.copy_(x)
        st = dict(case=c, logits=logits)
        st["bias"] = (torch.rand(E, generator=g, device="cuda") - 0.5) * 0.1 if c["bias"] else None
        if c["train"]:
            st["dw"] = torch.randn((T, c["k"]), generator=g, device="cuda")
        return st
    if c["op"] == "experts":
        T, E, k, H = c["T"], c["E"], c["k"], c["H"]
        pop = torch.rand(E, generator=g, device="cuda")
        score = torch.rand((T, E), generator=g, device="cuda") + pop
        order = torch.sort(score, dim=1, descending=True, stable=True)[1]
        ids = order[:, :min(k, E)].to(torch.int32)
        if k > E:
            ids = torch.cat([ids, ids.new_full((T, k - E), -1)], 1)
        pad = torch.rand(T, generator=g, device="cuda") < 0.01
        ids = torch.where(pad[:, None], ids.new_full((), -1), ids).contiguous()
        w = torch.rand((T, k), generator=g, device="cuda")
        w = torch.where(ids >= 0, w / w.sum(1, keepdim=True), w.new_zeros(())).contiguous()
        st = dict(case=c, ids=ids, w=w, x=_randn(g, T, H, 1.0), ys=_randn(g, T * k, H, 0.5))
        if c["train"]:
            st["dy"] = _randn(g, T, H, 1e-3)
            st["dxs"] = _randn(g, T * k, H, 1e-3)
        return st
    if c["op"] in ("fp8", "fp8_experts"):
        M, N, K = c["M"], c["N"], c["K"]
        st = dict(case=c, x=_randn(g, M, K, 1.0, outliers=True))
        if c["op"] == "fp8":
            w = torch.randn((N, K), generator=g, device="cuda") * 0.02
            q, s = _quantize_weights(w[None])
            st["spans"] = [(0, M)]
            st["offsets"] = None
        else:
            E = c["E"]
            w = torch.randn((E, N, K), generator=g, device="cuda") * 0.02
            q, s = _quantize_weights(w)
            off = _counts(g, M, E)
            h = off.tolist()
            st["spans"] = [(h[i], h[i + 1]) for i in range(E)]
            st["offsets"] = off.to(torch.int32)
        st["wq"], st["ws"] = q, s                                   # [E, N, K], [E, N/128, K/128]
        if c["train"]:
            st["wtq"] = _pitch16(q.view(torch.uint8).transpose(1, 2)
                                 .contiguous().view(torch.float8_e4m3fn))   # the same weights, [E, K, N]
            st["wts"] = s.transpose(1, 2).contiguous()
            st["dy"] = _randn(g, M, N, 1e-3)
        return st
    T, V, H = c["T"], c["V"], c["H"]
    # Token frequencies fall like 1 / rank, as in text; ranks are spread over the vocabulary.
    cdf = torch.cumsum(1.0 / (torch.arange(V, device="cuda", dtype=torch.float64) + 2.7), 0)
    rank = torch.searchsorted(cdf, torch.rand(T, generator=g, device="cuda", dtype=torch.float64) * cdf[-1])
    step = 48271
    while math.gcd(step, V) != 1:
        step += 2
    tokens = rank.clamp(max=V - 1) * step % V
    return dict(case=c, tokens=tokens, table=_randn(g, V, H, 0.02), dy=_randn(g, T, H, 1e-3))


# -------------------------------------------------------------- operators

def run(state):
    c = state["case"]
    return {"route": _route, "experts": _experts, "fp8": _fp8, "fp8_experts": _fp8, "embed": _embed}[c["op"]](state, c)


def _dg():
    import invariant_deterministic_gemm_gb300 as dg
    return dg


def _route(st, c):
    if own:
        dg = _dg()
        kw = dict(score=c["score"], renormalize=c["renorm"], scale=c["scale"])
        w, ids = dg.det_moe_route(st["logits"], c["k"], bias=st["bias"], n_groups=c["groups"],
                                  top_groups=c["top_groups"], **kw)
        if not c["train"]:
            return {"weights": w, "ids": ids}
        return {"weights": w, "ids": ids, "dlogits": dg.det_moe_route_bwd(st["dw"], st["logits"], ids, **kw)}
    k, E, G = c["k"], c["E"], c["groups"]
    x = st["logits"].double()        # values next to the border of the choice: 64 bits
    ok = x > -math.inf
    if c["score"] == "softmax":
        top = torch.where(ok, x, x.new_full((), -math.inf)).amax(1, keepdim=True)
        e = torch.where(ok, torch.exp(x - top), x.new_zeros(()))
        p = torch.where(ok, e / e.sum(1, keepdim=True), x.new_zeros(()))
        choice = x if st["bias"] is None and G == 1 else p
    else:
        p = torch.where(ok, 1.0 / (1.0 + torch.exp(-x)), x.new_zeros(()))
        choice = p
    if st["bias"] is not None:
        choice = choice + st["bias"].double()
    choice = torch.where(ok, choice, x.new_full((), -math.inf))
    if G > 1:
        best = torch.sort(choice.reshape(-1, G, E // G), dim=2, descending=True)[0][:, :, :2]
        some = best[:, :, 0] > -math.inf
        total = torch.where(best > -math.inf, best, best.new_zeros(())).sum(2)
        total = torch.where(some, total, total.new_full((), -math.inf))
        kept = torch.sort(total, dim=1, descending=True, stable=True)[1][:, :c["top_groups"]]
        keep = torch.zeros_like(total).scatter(1, kept, 1.0).bool().repeat_interleave(E // G, 1)
        choice = torch.where(keep, choice, choice.new_full((), -math.inf))
    val, ids = torch.sort(choice, dim=1, descending=True, stable=True)
    chosen = val[:, :k] > -math.inf
    ids = ids[:, :k]
    w = torch.where(chosen, p.gather(1, ids), p.new_zeros(()))
    eps = SIGMOID_EPS if c["score"] == "sigmoid" else 0.0
    S = w.sum(1, keepdim=True) + eps
    S = torch.where(chosen.any(1, keepdim=True), S, S.new_ones(()))
    wr = w / S if c["renorm"] else w
    out = {"weights": (wr * c["scale"]).float(), "ids": torch.where(chosen, ids, ids.new_full((), -1)).to(torch.int32)}
    if c["train"]:
        gr = torch.where(chosen, st["dw"].double() * c["scale"], w.new_zeros(()))
        if c["renorm"]:
            gr = (gr - (gr * wr).sum(1, keepdim=True)) / S
        gd = torch.zeros_like(p).scatter_add(1, ids, torch.where(chosen, gr, gr.new_zeros(())))
        if c["score"] == "softmax":
            dl = p * (gd - (gd * p).sum(1, keepdim=True))
        else:
            dl = gd * p * (1.0 - p)
        out["dlogits"] = dl.to(st["logits"].dtype)
    return out


def _experts(st, c):
    T, E, k = c["T"], c["E"], c["k"]
    if own:
        dg = _dg()
        offsets, rows, slots = dg.det_moe_dispatch(st["ids"], E)
        out = {"offsets": offsets, "rows": rows, "slots": slots,
               "xs": dg.det_moe_gather(st["x"], rows, k),
               "y": dg.det_moe_combine(st["ys"], slots, st["w"])}
        if c["train"]:
            out["dys"], out["dw"] = dg.det_moe_combine_bwd(st["dy"], st["ys"], rows, slots, st["w"])
            out["dx"] = dg.det_moe_combine(st["dxs"], slots)
        return out
    ids = st["ids"].reshape(-1).long()
    key = torch.where(ids >= 0, ids, ids.new_full((), E))
    order = torch.sort(key, stable=True)[1]
    bounds = torch.arange(E + 1, device="cuda")
    offsets = (key[None, :] < bounds[:, None]).sum(1).to(torch.int32)
    used = torch.arange(T * k, device="cuda") < offsets[-1]
    rows = torch.where(used, order, order.new_full((), -1))
    slots = torch.empty_like(order).scatter_(0, order, torch.arange(T * k, device="cuda"))
    slots = torch.where(ids >= 0, slots, slots.new_full((), -1))
    src = (rows.clamp(min=0) // k)
    zero = torch.zeros((), device="cuda")
    xs = torch.where(used[:, None], st["x"][src], zero.to(torch.bfloat16))
    at = slots.clamp(min=0).reshape(T, k)
    hit = (slots >= 0).reshape(T, k)

    def combined(v, w):
        acc = torch.zeros((T, v.shape[1]), device="cuda")
        for j in range(k):
            r = torch.where(hit[:, j, None], v[at[:, j]].float(), zero)
            acc = acc + (r if w is None else w[:, j, None] * r)
        return acc.to(torch.bfloat16)

    out = {"offsets": offsets, "rows": rows.to(torch.int32), "slots": slots.reshape(T, k).to(torch.int32), "xs": xs,
           "y": combined(st["ys"], st["w"])}
    if c["train"]:
        flat_w = st["w"].reshape(-1)[rows.clamp(min=0)]
        dyr = st["dy"][src].float()
        out["dys"] = torch.where(used[:, None], flat_w[:, None] * dyr, zero).to(torch.bfloat16)
        dw = torch.empty((T, k), device="cuda")
        for j in range(k):
            dw[:, j] = torch.where(hit[:, j], (st["dy"].float() * st["ys"][at[:, j]].float()).sum(1), zero)
        out["dw"] = dw
        out["dx"] = combined(st["dxs"], None)
    return out


def _dequantized_rows(x):
    """x [M, K] quantised along K in blocks of 128, as the values it then stands for."""
    t = _blocks(x.float(), 1)
    amax = t.abs().amax(2, keepdim=True).clamp(min=AMAX_MIN)
    q = (t * E4M3_MAX / amax).to(torch.float8_e4m3fn).float()
    return (q * (amax / E4M3_MAX)).reshape(x.shape[0], -1)[:, :x.shape[1]]


def _dequantized_weights(q, s):
    t = q.float()
    return t * s.repeat_interleave(BLOCK, 0)[:t.shape[0]].repeat_interleave(BLOCK, 1)[:, :t.shape[1]]


def _fp8(st, c):
    out_t = torch.float32 if c["out"] == "fp32" else torch.bfloat16
    if own:
        dg = _dg()
        off = st["offsets"]
        xq, xs = dg.det_fp8_quantize_rows(st["x"])
        if off is None:
            out = {"y": dg.det_fp8_gemm(xq, xs, st["wq"][0], st["ws"][0])}
        else:
            out = {"y": dg.det_fp8_gemm_grouped(xq, xs, st["wq"], st["ws"], off)}
        if c["train"]:
            gq, gs = dg.det_fp8_quantize_rows(st["dy"])
            if off is None:
                out["dx"] = dg.det_fp8_gemm(gq, gs, st["wtq"][0], st["wts"][0])
            else:
                out["dx"] = dg.det_fp8_gemm_grouped(gq, gs, st["wtq"], st["wts"], off)
            gt, gts = dg.det_fp8_quantize_cols(st["dy"], off)
            xt, xts = dg.det_fp8_quantize_cols(st["x"], off)
            out["dw"] = dg.det_fp8_gemm_wgrad(gt, gts, xt, xts, off, out_dtype=out_t)
        return out
    M, N, K, E = c["M"], c["N"], c["K"], len(st["spans"])
    y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    out = {"y": y}
    xd = _dequantized_rows(st["x"])
    if c["train"]:
        gd = _dequantized_rows(st["dy"])
        dx = out["dx"] = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
        dw = out["dw"] = torch.empty((N, K) if st["offsets"] is None else (E, N, K), dtype=out_t, device="cuda")
    for e, (lo, hi) in enumerate(st["spans"]):
        if hi > lo:
            w = _dequantized_weights(st["wq"][e], st["ws"][e])
            y[lo:hi] = (xd[lo:hi] @ w.T).to(torch.bfloat16)
            if c["train"]:
                dx[lo:hi] = (gd[lo:hi] @ w).to(torch.bfloat16)
        if c["train"]:
            xt = _dequantized_rows(st["x"][lo:hi].T.contiguous())
            gt = _dequantized_rows(st["dy"][lo:hi].T.contiguous())
            (dw if st["offsets"] is None else dw[e]).copy_(gt @ xt.T)
    return out


def _embed(st, c):
    grad_t = torch.float32 if c["grad"] == "fp32" else torch.bfloat16
    if own:
        dg = _dg()
        return {"out": dg.det_embedding(st["tokens"], st["table"], c["scale"]),
                "dtable": dg.det_embedding_grad(st["dy"], st["tokens"], c["V"], c["scale"], out_dtype=grad_t)}
    out = (st["table"][st["tokens"]].float() * c["scale"]).to(torch.bfloat16)
    d = torch.zeros((c["V"], c["H"]), device="cuda")
    d.index_add_(0, st["tokens"], st["dy"].float())
    return {"out": out, "dtable": (d * c["scale"]).to(grad_t)}


# ------------------------------------------------------------------ exact

def _e4m3(v):
    """v (64 bits) rounded to the nearest e4m3 value, ties to even."""
    _, ex = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), torch.clamp(ex - 1, min=-6) - 3)
    return torch.clamp(torch.round(v / step) * step, -E4M3_MAX, E4M3_MAX)


def _exact_rows(x):
    out = torch.empty(x.shape, dtype=torch.float64, device="cuda")
    for k0 in range(0, x.shape[1], BLOCK):
        v = x[:, k0:k0 + BLOCK].double()
        if v.numel() == 0:
            continue
        amax = torch.clamp(v.abs().max(1, keepdim=True)[0], min=AMAX_MIN)
        out[:, k0:k0 + BLOCK] = _e4m3(v * E4M3_MAX / amax) * amax / E4M3_MAX
    return out


def _exact_cols(x):
    out = torch.empty(x.shape, dtype=torch.float64, device="cuda")
    for r0 in range(0, x.shape[0], BLOCK):
        v = x[r0:r0 + BLOCK].double()
        amax = torch.clamp(v.abs().max(0, keepdim=True)[0], min=AMAX_MIN)
        out[r0:r0 + BLOCK] = _e4m3(v * E4M3_MAX / amax) * amax / E4M3_MAX
    return out


def _exact_weights(q, s):
    w = q.double()
    for n0 in range(0, w.shape[0], BLOCK):
        for k0 in range(0, w.shape[1], BLOCK):
            w[n0:n0 + BLOCK, k0:k0 + BLOCK] *= s[n0 // BLOCK, k0 // BLOCK].double()
    return w


def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["op"] == "route":
        return _exact_route(st, c)
    if c["op"] == "experts":
        T, E, k, H = c["T"], c["E"], c["k"], c["H"]
        ids = st["ids"].cpu().reshape(-1).tolist()
        lists = [[] for _ in range(E)]
        for i, e in enumerate(ids):
            if 0 <= e < E:
                lists[e].append(i)
        rows, offsets = [], [0]
        for l in lists:
            rows += l
            offsets.append(len(rows))
        n = len(rows)
        slots = [-1] * (T * k)
        for r, i in enumerate(rows):
            slots[i] = r
        ri = torch.tensor(rows, dtype=torch.int64, device="cuda")
        rows = rows + [-1] * (T * k - n)
        out = {"offsets": torch.tensor(offsets, dtype=torch.int32), "rows": torch.tensor(rows, dtype=torch.int32),
               "slots": torch.tensor(slots, dtype=torch.int32).reshape(T, k)}
        tok = torch.div(ri, k, rounding_mode="floor")
        w = st["w"].double().reshape(-1)
        xs = torch.zeros((T * k, H), dtype=torch.float64, device="cuda")
        xs[:n] = st["x"].double()[tok]
        y = torch.zeros((T, H), dtype=torch.float64, device="cuda")
        y.index_add_(0, tok, w[ri, None] * st["ys"][:n].double())
        out["xs"], out["y"] = xs, y
        if c["train"]:
            dyr = st["dy"].double()[tok]
            dys = torch.zeros((T * k, H), dtype=torch.float64, device="cuda")
            dys[:n] = w[ri, None] * dyr
            dw = torch.zeros(T * k, dtype=torch.float64, device="cuda")
            dw[ri] = (dyr * st["ys"][:n].double()).sum(1)
            dx = torch.zeros((T, H), dtype=torch.float64, device="cuda")
            dx.index_add_(0, tok, st["dxs"][:n].double())
            out.update(dys=dys, dw=dw.reshape(T, k), dx=dx)
        return out
    if c["op"] in ("fp8", "fp8_experts"):
        M, N, K, E = c["M"], c["N"], c["K"], len(st["spans"])
        out = {"y": torch.empty((M, N), dtype=torch.float64, device="cuda")}
        if c["train"]:
            out["dx"] = torch.empty((M, K), dtype=torch.float64, device="cuda")
            dw = torch.zeros((E, N, K), dtype=torch.float64, device="cuda")
            out["dw"] = dw[0] if st["offsets"] is None else dw
        for e, (lo, hi) in enumerate(st["spans"]):
            if hi == lo:
                continue
            w = _exact_weights(st["wq"][e], st["ws"][e])
            out["y"][lo:hi] = _exact_rows(st["x"][lo:hi]) @ w.T
            if c["train"]:
                out["dx"][lo:hi] = _exact_rows(st["dy"][lo:hi]) @ w
                dw[e] = _exact_cols(st["dy"][lo:hi]).T @ _exact_cols(st["x"][lo:hi])
        return out
    out = st["table"].double()[st["tokens"]] * c["scale"]
    d = torch.zeros((c["V"], c["H"]), dtype=torch.float64, device="cuda")
    d.index_add_(0, st["tokens"], st["dy"].double() * c["scale"])
    return {"out": out, "dtable": d}


def _exact_route(st, c):
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    l = st["logits"].double()
    live = torch.isfinite(l)
    neg = torch.full_like(l, -math.inf)
    z = torch.zeros_like(l)
    if c["score"] == "softmax":
        score = torch.where(live, torch.nan_to_num(torch.softmax(torch.where(live, l, neg), 1), nan=0.0), z)
        rank = score if st["bias"] is not None or G > 1 else l
    else:
        score = torch.where(live, torch.sigmoid(torch.where(live, l, z)), z)
        rank = score
    if st["bias"] is not None:
        rank = rank + st["bias"].double()[None, :]
    rank = torch.where(live, rank, neg)
    if G > 1:
        r = rank.reshape(T, G, E // G)
        first, at = r.max(2)
        second = r.scatter(2, at[:, :, None], -math.inf).max(2)[0]
        group = torch.where(second > -math.inf, first + second, first)
        left = torch.zeros((T, G), dtype=torch.bool, device="cuda")
        for _ in range(c["top_groups"]):
            cand = torch.where(left, torch.full_like(group, -math.inf), group)
            m = cand.max(1, keepdim=True)[0]
            pick = ((cand == m) & ~left).float().argmax(1)
            left[torch.arange(T, device="cuda"), pick] = True
        rank = torch.where(left[:, :, None].expand(T, G, E // G).reshape(T, E), rank, neg)
    ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    w = torch.zeros((T, k), dtype=torch.float64, device="cuda")
    t = torch.arange(T, device="cuda")
    for j in range(k):
        m = rank.max(1, keepdim=True)[0]
        pick = (rank == m).float().argmax(1)
        got = m[:, 0] > -math.inf
        ids[:, j] = torch.where(got, pick, -1).to(torch.int32)
        w[:, j] = torch.where(got, score[t, pick], 0.0)
        rank[t, pick] = -math.inf
    got = ids >= 0
    S = w.sum(1, keepdim=True) + (SIGMOID_EPS if c["score"] == "sigmoid" else 0.0)
    S[~got.any(1)] = 1.0
    out = {"weights": (w / S if c["renorm"] else w) * c["scale"], "ids": ids}
    if c["train"]:
        # Through the Jacobian of the weights with respect to the chosen scores, then of the scores.
        up = torch.where(got, st["dw"].double() * c["scale"], 0.0)
        if c["renorm"]:
            up = up / S - (up * w).sum(1, keepdim=True) / (S * S)
            up = torch.where(got, up, 0.0)
        d = torch.zeros_like(l)
        for j in range(k):
            d[t, ids[:, j].clamp(min=0).long()] += up[:, j]
        if c["score"] == "softmax":
            out["dlogits"] = score * d - score * (score * d).sum(1, keepdim=True)
        else:
            out["dlogits"] = score * (1.0 - score) * d
    return out
