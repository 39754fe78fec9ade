"""Performance cases of the attention operators.

Each case runs one operator the way a program uses it: rotary positions with
their gradient, appending rotated keys and values to a paged cache, attention
of one new token over that cache, and attention of packed sequences with a
sliding window and first tokens that stay visible, forward and backward.
``run`` computes the operator in elementary torch operations in FP32, or,
when ``own`` is set, calls the package's operators; ``exact`` computes it in
64 bits from the definition.
"""
import math

import torch

own = False

ROPE_BASE = 10000.0
BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32


# ------------------------------------------------------------------ cases

def listed():
    return [
        # A decode step of 17 sequences: the QKV projection's 12288 columns as 32 heads of 128, one new row each in the cache.
        dict(name="append_decode", op="append", T=17, H=32, KV=32, D=128, rot=128, inter=False, page=16, P=8192),
        # A prompt's keys and values on their way to the cache, eight shared heads.
        dict(name="append_prompt", op="append", T=8192, H=32, KV=8, D=128, rot=128, inter=False, page=64, P=131072),
        # Rotation in a training step, forward and gradient: odd sizes, half of a head's columns, neighbouring pairs.
        dict(name="rope_train_odd", op="rope", T=4099, H=12, KV=4, D=80, rot=40, inter=True, P=8192),
        # One user's next token after a page of text.
        dict(name="decode_one", op="decode", B=1, L=1021, H=32, KV=32, D=128, page=16, window=0, sinks=0),
        # A serving batch with ragged contexts up to 8192, a padded slot among them.
        dict(name="decode_batch", op="decode", B=64, L=8192, H=32, KV=8, D=128, page=16, window=0, sinks=0),
        # A larger batch of a model with a sliding window and sinks, heads of 64.
        dict(name="decode_window", op="decode", B=96, L=16384, H=64, KV=8, D=64, page=32, window=1024, sinks=4),
        # Two very long contexts: the cache's length is all the parallelism there is.
        dict(name="decode_long", op="decode", B=2, L=262144, H=32, KV=8, D=128, page=64, window=0, sinks=0),
        # A short prompt.
        dict(name="prompt_short", op="attn", T=333, N=1, past=0, H=32, KV=32, D=128, window=0, sinks=0, train=False),
        # Chunks of four prompts whose first parts are in the cache already.
        dict(name="prompt_chunks", op="attn", T=2048, N=4, past=6144, H=32, KV=8, D=128, window=0, sinks=0, train=False),
        # A long document through a layer with a window and sinks.
        dict(name="prompt_window", op="attn", T=16384, N=1, past=0, H=16, KV=4, D=128, window=1024, sinks=4, train=False),
        # A training step's 8192 tokens packed from five documents, forward and backward.
        dict(name="train_packed", op="attn", T=8192, N=5, past=0, H=32, KV=8, D=128, window=0, sinks=0, train=True),
        # A small model's training step: odd sizes, heads of 80, a window that is no multiple of anything.
        dict(name="train_window_odd", op="attn", T=2047, N=3, past=0, H=12, KV=4, D=80, window=257, sinks=5, train=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "rope", "decode", "attn", "attn"])
    KV = rng.choice([1, 2, 4, 8])
    H = KV * rng.choice([1, 2, 3, 4, 8])
    D = 8 * rng.randint(4, 16)
    if op in ("append", "rope"):
        c = dict(op=op, T=_log(rng, 1, 8192), H=H, KV=KV, D=D, rot=8 * rng.randint(1, D // 8), inter=rng.random() < 0.5,
                 P=_log(rng, 256, 131072))
        if op == "append":
            c["page"] = 8 * _log(rng, 1, 32)
        return c
    window = _log(rng, 1, 4096) if rng.random() < 0.5 else 0
    sinks = rng.randint(0, 20) if window else 0
    if op == "decode":
        B = _log(rng, 1, 128)
        return dict(op=op, B=B, L=_log(rng, 1, min(262144, 524288 // B)), H=H, KV=KV, D=D, page=8 * _log(rng, 1, 32),
                    window=window, sinks=sinks)
    past = _log(rng, 1, 4096) if rng.random() < 0.3 else 0
    T = _log(rng, 1, min(8192, int(math.sqrt(2e9 / H)) - past // 2))       # fewer pairs than the largest listed case
    N = rng.randint(1, min(8, T))
    return dict(op=op, T=T, N=N, past=past, H=H, KV=KV, D=D, window=window, sinks=sinks, train=past == 0 and rng.random() < 0.6)


def _parts(total, n):
    """`total` in n uneven parts of at least one."""
    w = [1 + 3 * ((5 * i + 2) % 7) for i in range(n)]
    edges = [i + (total - n) * sum(w[:i]) // sum(w) for i in range(n + 1)]
    return [edges[i + 1] - edges[i] for i in range(n)]


def _contexts(c):
    """Lengths of a decode case's sequences: the longest first, then ragged, from eight sequences on one of them empty."""
    B, L = c["B"], c["L"]
    n = [max(1, L * (2 * B - (3 * i) % B - (i % 2) * (B // 2)) // (2 * B) - (i % 3 if i else 0)) for i in range(B)]
    if B >= 8:
        n[B // 2] = 0
    return n


def _seen(n, window, sinks):
    """How many of n keys the last token sees."""
    return n if not window or n <= window else window + min(sinks, n - window)


def _pairs(c):
    total = 0
    for q, past in zip(_parts(c["T"], c["N"]), _pasts(c)):
        for i in (range(past + 1, past + q + 1)):
            total += _seen(i, c["window"], c["sinks"])
    return total


def _pasts(c):
    return _parts(c["past"], c["N"]) if c["past"] >= c["N"] else [c["past"]] + [0] * (c["N"] - 1)


def work(case):
    c = case
    H, KV, D = c["H"], c["KV"], c["D"]
    if c["op"] == "append":
        T = c["T"]
        return {"bytes": T * (4 * H * D + 8 * KV * D + 8) + min(T, c["P"]) * c["rot"] * 4, "flops": 3.0 * T * (H + KV) * c["rot"]}
    if c["op"] == "rope":
        T = c["T"]
        return {"bytes": T * (8 * (H + KV) * D + 4) + min(T, c["P"]) * c["rot"] * 4, "flops": 6.0 * T * (H + KV) * c["rot"]}
    if c["op"] == "decode":
        keys = sum(_seen(n, c["window"], c["sinks"]) for n in _contexts(c))
        return {"bytes": 4 * keys * KV * D + 4 * c["B"] * H * D + 4 * keys // c["page"] + 4 * c["B"], "flops": 4.0 * keys * H * D}
    T, S = c["T"], c["T"] + c["past"]
    b = 4 * T * H * D + 4 * S * KV * D + 4 * T * H
    f = 4.0 * _pairs(c) * H * D
    if c["train"]:
        b += 4 * T * H * D + 4 * S * KV * D       # dout, dq; dk, dv
        f += 10.0 * _pairs(c) * H * D
    return {"bytes": b, "flops": f}


# ----------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 2654435761 % (1 << 62) + 29)


def _tables(P, rot):
    """cos and sin [P, rot / 2] FP32 of position times base^(-2i / rot), the angle in 64 bits."""
    freq = ROPE_BASE ** (-torch.arange(0, rot, 2, device="cuda", dtype=F64) / rot)
    angle = torch.arange(P, device="cuda", dtype=F64)[:, None] * freq
    return torch.cos(angle).float(), torch.sin(angle).float()


def _qkv(g, T, H, KV, D):
    """One projection's output [T, (H + 2 KV) D] as its three views; heads differ in how sharply they look."""
    x = torch.randn((T, H + 2 * KV, D), generator=g, device="cuda")
    x[:, :H] *= 0.5 + 2.0 * torch.rand((H, 1), generator=g, device="cuda")
    x = x.to(BF16)
    return x[:, :H], x[:, H:H + KV], x[:, H + KV:]


def _bounds(lengths):
    n = torch.tensor([0] + lengths, dtype=torch.int64)
    return torch.cumsum(n, 0).to(I32).cuda()


def _roll(v, seed):
    k = int(seed) % len(v)
    return v[k:] + v[:k]


def prepare(case, seed):
    c, g = case, _gen(seed)
    H, KV, D = c["H"], c["KV"], c["D"]
    if c["op"] in ("append", "rope"):
        T, P = c["T"], c["P"]
        q, k, v = _qkv(g, T, H, KV, D)
        cos, sin = _tables(P, c["rot"])
        st = dict(case=c, q=q, k=k, v=v, cos=cos, sin=sin)
        first = int(torch.randint(0, max(1, P - T), (1,), generator=g, device="cuda"))
        st["pos"] = ((torch.arange(T, device="cuda") + first) % P).to(I32)
        if c["op"] == "rope":
            dq, dk, _ = _qkv(g, T, H, KV, D)
            st["dq"], st["dk"] = (dq * 1e-3).contiguous(), (dk * 1e-3).contiguous()
            return st
        pages = -(-T // c["page"]) + 3
        slots = torch.randperm(pages, generator=g, device="cuda")[:, None] * c["page"] + torch.arange(c["page"], device="cuda")
        slots = slots.reshape(-1)[:T]
        st["slots"] = torch.where(torch.rand(T, generator=g, device="cuda") < 0.02, slots.new_full((), -1), slots).to(I32)
        st["kc"] = torch.randn((pages, c["page"], KV, D), generator=g, device="cuda").to(BF16)
        st["vc"] = torch.randn((pages, c["page"], KV, D), generator=g, device="cuda").to(BF16)
        return st
    if c["op"] == "decode":
        n = _roll(_contexts(c), seed)
        most = max(1, -(-max(n) // c["page"]))
        held = [-(-x // c["page"]) for x in n]
        lengths, held_t = torch.tensor(n, dtype=I32).cuda(), torch.tensor(held).cuda()
        pages = max(1, sum(held))
        perm = torch.randperm(pages, generator=g, device="cuda").to(I32)
        at = (torch.cumsum(held_t, 0) - held_t)[:, None] + torch.arange(most, device="cuda")
        table = torch.where(torch.arange(most, device="cuda") < held_t[:, None], perm[at.clamp(max=pages - 1)], perm.new_full((), -1))
        q, _, _ = _qkv(g, c["B"], H, KV, D)
        return dict(case=c, q=q, table=table.contiguous(), lengths=lengths,
                    kc=torch.randn((pages, c["page"], KV, D), generator=g, device="cuda").to(BF16),
                    vc=torch.randn((pages, c["page"], KV, D), generator=g, device="cuda").to(BF16))
    qn, past = _roll(_parts(c["T"], c["N"]), seed), _roll(_pasts(c), seed)
    q, k, v = _qkv(g, c["T"], H, KV, D)
    st = dict(case=c, q=q, k=k, v=v, bounds=_bounds(qn), k_bounds=None, spans=qn, k_spans=qn)
    if c["past"]:
        _, st["k"], st["v"] = _qkv(g, c["T"] + c["past"], 0, KV, D)
        st["k_spans"] = [a + b for a, b in zip(qn, past)]
        st["k_bounds"] = _bounds(st["k_spans"])
    if c["train"]:
        st["dout"] = (torch.randn((c["T"], H, D), generator=g, device="cuda") * 1e-3).to(BF16)
    return st


# -------------------------------------------------------------- operators

def run(state):
    c = state["case"]
    return {"append": _append, "rope": _rope, "decode": _decode, "attn": _attn}[c["op"]](state, c)


def _dg():
    import invariant_deterministic_gemm_gb300 as dg
    return dg


def _rotated(x, cos, sin, pos, inter, inverse=False):
    half = cos.shape[1]
    xf, p = x.float(), pos.long()
    co, si = cos[p][:, None], sin[p][:, None]
    if inverse:
        si = -si
    if inter:
        a, b = xf[..., 0:2 * half:2], xf[..., 1:2 * half:2]
        r = torch.stack([a * co - b * si, b * co + a * si], -1).flatten(-2)
    else:
        a, b = xf[..., :half], xf[..., half:2 * half]
        r = torch.cat([a * co - b * si, b * co + a * si], -1)
    return torch.cat([r, xf[..., 2 * half:]], -1).to(BF16)


def _rope(st, c):
    if own:
        dg = _dg()
        a = (st["cos"], st["sin"], st["pos"])
        return {"q": dg.det_rope(st["q"], *a, interleaved=c["inter"]), "k": dg.det_rope(st["k"], *a, interleaved=c["inter"]),
                "dq": dg.det_rope(st["dq"], *a, interleaved=c["inter"], inverse=True),
                "dk": dg.det_rope(st["dk"], *a, interleaved=c["inter"], inverse=True)}
    a = (st["cos"], st["sin"], st["pos"], c["inter"])
    return {"q": _rotated(st["q"], *a), "k": _rotated(st["k"], *a), "dq": _rotated(st["dq"], *a, True),
            "dk": _rotated(st["dk"], *a, True)}


def _append(st, c):
    kc, vc = st["kc"], st["vc"]
    if own:
        q = _dg().det_kv_append(st["q"], st["k"], st["v"], st["cos"], st["sin"], st["pos"], st["slots"], kc, vc,
                                interleaved=c["inter"])
        return {"q": q, "kc": kc, "vc": vc}
    a = (st["cos"], st["sin"], st["pos"], c["inter"])
    kept = torch.nonzero(st["slots"] >= 0)[:, 0]
    to = st["slots"][kept].long()
    kc.view(-1, *kc.shape[2:])[to] = _rotated(st["k"], *a)[kept]
    vc.view(-1, *vc.shape[2:])[to] = st["v"][kept]
    return {"q": _rotated(st["q"], *a), "kc": kc, "vc": vc}


def _decode(st, c):
    window, sinks = c["window"], c["sinks"]
    if own:
        return {"out": _dg().det_attn_decode(st["q"], st["kc"], st["vc"], st["table"], st["lengths"], window=window or None, sinks=sinks)}
    B, KV, D = c["B"], c["KV"], c["D"]
    at = st["table"].clamp(min=0).long()
    n = st["lengths"].long()[:, None]
    j = torch.arange(at.shape[1] * c["page"], device="cuda")[None]
    vis = j < n
    if window:
        vis = vis & ((j >= n - window) | (j < sinks))
    k = st["kc"][at].reshape(B, -1, KV, D).permute(0, 2, 3, 1).float()
    q = st["q"].reshape(B, KV, -1, D).float()
    s = (q @ k) * (1.0 / math.sqrt(D))
    del k
    vis = vis[:, None, None]
    s = torch.where(vis, s, s.new_full((), -math.inf))
    top = s.amax(3, keepdim=True)
    p = torch.exp(s - torch.where(top > -math.inf, top, top.new_zeros(())))
    p = p / p.sum(3, keepdim=True).clamp(min=1e-38)
    v = st["vc"][at].reshape(B, -1, KV, D).permute(0, 2, 1, 3).float()
    return {"out": (p @ v).reshape(B, -1, D).to(BF16)}


def _visible(st, c):
    """[T, S]: which keys each query sees."""
    T, S = st["q"].shape[0], st["k"].shape[0]
    qb = st["bounds"].long()
    kb = qb if st["k_bounds"] is None else st["k_bounds"].long()
    t, s = torch.arange(T, device="cuda"), torch.arange(S, device="cuda")
    qs, ks = (t[:, None] >= qb[None, 1:]).sum(1), (s[:, None] >= kb[None, 1:]).sum(1)      # the sequence of each row
    top = c["N"] - 1
    qi = t - qb[qs.clamp(max=top) + 1] + kb[qs.clamp(max=top) + 1] - kb[qs.clamp(max=top)]   # position in its sequence
    ki = s - kb[ks.clamp(max=top)]
    vis = (qs[:, None] == ks) & (ki <= qi[:, None])
    if c["window"]:
        vis = vis & ((ki > qi[:, None] - c["window"]) | (ki < c["sinks"]))
    return vis


def _attn(st, c):
    H, KV, D = c["H"], c["KV"], c["D"]
    if own:
        dg = _dg()
        kw = dict(k_bounds=st["k_bounds"], window=c["window"] or None, sinks=c["sinks"])
        out, lse = dg.det_attn(st["q"], st["k"], st["v"], st["bounds"], **kw)
        r = {"out": out, "lse": lse}
        if c["train"]:
            r["dq"], r["dk"], r["dv"] = dg.det_attn_bwd(st["dout"], st["q"], st["k"], st["v"], out, lse, st["bounds"], **kw)
        return r
    T, S, G, scale = c["T"], st["k"].shape[0], H // KV, 1.0 / math.sqrt(D)
    vis = _visible(st, c)
    q = st["q"].permute(1, 0, 2).reshape(KV, G * T, D).float()
    k, v = st["k"].permute(1, 0, 2).float(), st["v"].permute(1, 0, 2).float()
    s = (q @ k.transpose(1, 2)).reshape(KV, G, T, S).mul_(scale)
    s = s.masked_fill_(~vis, -math.inf)
    top = s.amax(3, keepdim=True)
    top = torch.where(top > -math.inf, top, top.new_zeros(()))
    p = s.sub_(top).exp_()
    total = p.sum(3, keepdim=True)
    r = {"lse": (top + torch.log(total)).reshape(H, T)}
    p = p.div_(total.clamp(min=1e-38)).reshape(KV, G * T, S)
    r["out"] = (p @ v).reshape(H, T, D).permute(1, 0, 2).to(BF16)
    if c["train"]:
        do = st["dout"].permute(1, 0, 2).reshape(KV, G * T, D).float()
        r["dv"] = (p.transpose(1, 2) @ do).permute(1, 0, 2).to(BF16)
        dp = do @ v.transpose(1, 2)
        ds = dp.sub_((p * dp).sum(2, keepdim=True)).mul_(p).mul_(scale)
        r["dq"] = (ds @ k).reshape(H, T, D).permute(1, 0, 2).to(BF16)
        r["dk"] = (ds.transpose(1, 2) @ q).permute(1, 0, 2).to(BF16)
    return r


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    c = case
    st = prepare(c, seed)
    if c["op"] == "append":
        K, V = st["kc"].double(), st["vc"].double()
        for x, cache in ((_turn(st["k"], st, c, 1.0), K), (st["v"].double(), V)):
            flat = cache.view(-1, *cache.shape[2:])
            keep = st["slots"] >= 0
            flat[st["slots"][keep].long()] = x[keep]
        return {"q": _turn(st["q"], st, c, 1.0), "kc": K, "vc": V}
    if c["op"] == "rope":
        return {n: _turn(st[n], st, c, f) for n, f in (("q", 1.0), ("k", 1.0), ("dq", -1.0), ("dk", -1.0))}
    if c["op"] == "decode":
        return {"out": _exact_decode(st, c)}
    return _exact_attn(st, c)


def _turn(x, st, c, direction):
    """Each pair as a complex number, times cos + i sin (its conjugate for the gradient)."""
    w = torch.complex(st["cos"].double(), direction * st["sin"].double())[st["pos"].long()][:, None]
    y, R = x.double().clone(), c["rot"]
    first = slice(0, R, 2) if c["inter"] else slice(0, R // 2)
    second = slice(1, R, 2) if c["inter"] else slice(R // 2, R)
    z = torch.complex(y[..., first].clone(), y[..., second].clone()) * w
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_decode(st, c):
    B, H, D, page = c["B"], c["H"], c["D"], c["page"]
    out = torch.zeros((B, H, D), dtype=F64, device="cuda")
    for b, n in enumerate(st["lengths"].tolist()):
        if not n:
            continue
        seen = list(range(n)) if not c["window"] or n <= c["window"] + c["sinks"] else None
        seen = torch.arange(n, device="cuda") if seen is not None else torch.cat(
            [torch.arange(c["sinks"], device="cuda"), torch.arange(n - c["window"], n, device="cuda")])
        at = st["table"][b].long()[seen // page] * page + seen % page
        for h in range(c["KV"]):
            k, v = (st[x].reshape(-1, c["KV"], D)[at, h].double() for x in ("kc", "vc"))
            g = slice(h * (H // c["KV"]), (h + 1) * (H // c["KV"]))
            out[b, g] = torch.softmax(st["q"][b, g].double() @ k.T / math.sqrt(D), 1) @ v
    return out


def _exact_attn(st, c):
    T, S, H, KV, D, W = c["T"], st["k"].shape[0], c["H"], c["KV"], c["D"], c["window"]
    flops = (14 if c["train"] else 4) * H * D * sum(a * min(b, (W or b) + 2048) for a, b in zip(st["spans"], st["k_spans"]))
    if flops > 1.2e13:
        return None
    new = lambda *shape: torch.zeros(shape, dtype=F64, device="cuda")  # noqa: E731
    r = {"out": new(T, H, D), "lse": torch.full((H, T), -math.inf, dtype=F64, device="cuda")}
    if c["train"]:
        r.update(dq=new(T, H, D), dk=new(S, KV, D), dv=new(S, KV, D))
    scale, q0, k0 = D ** -0.5, 0, 0
    for nq, nk in zip(st["spans"], st["k_spans"]):
        for a in range(0, nq, 2048):                     # queries [a, b) of the sequence, and the keys that any of them sees
            b = min(a + 2048, nq)
            i = torch.arange(a, b, device="cuda") + nk - nq
            last = b + nk - nq
            lo = max(0, a + nk - nq - W + 1) if W else 0
            j = torch.cat([torch.arange(0, min(c["sinks"], lo), device="cuda"), torch.arange(lo, last, device="cuda")])
            hidden = j[None] > i[:, None]
            if W:
                hidden |= (i[:, None] - j[None] >= W) & (j[None] >= c["sinks"])
            rows, keys = slice(q0 + a, q0 + b), k0 + j
            for h in range(H):
                g = h // (H // KV)
                q, k, v = st["q"][rows, h].double(), st["k"][keys, g].double(), st["v"][keys, g].double()
                s = (q @ k.T * scale).masked_fill_(hidden, -math.inf)
                lse = torch.logsumexp(s, 1)
                p = torch.exp(s - lse[:, None])
                r["lse"][h, rows] = lse
                o = r["out"][rows, h] = p @ v
                if c["train"]:
                    do = st["dout"][rows, h].double()
                    ds = p * (do @ v.T - (do * o).sum(1, keepdim=True)) * scale
                    r["dq"][rows, h] = ds @ k
                    r["dk"][:, g].index_add_(0, keys, ds.T @ q)
                    r["dv"][:, g].index_add_(0, keys, p.T @ do)
        q0, k0 = q0 + nq, k0 + nk
    return r
