"""Routing, dispatch and combine on the GPU against 64-bit implementations
(tests/ops_ref.py): ids, orders and copies exactly, sums within bounds
derived from their number of FP32 roundings; rows that leave nothing to
choose, NaN and infinite logits, ties, one token, odd sizes, strides; and
bits that do not depend on the batch."""
import numpy as np
import pytest
import torch

import invariant_deterministic_gemm_gb300 as dg
import ops_ref as ref

pytestmark = pytest.mark.gpu
INF = float("inf")


def ok():
    assert dg.det_gemm_check() == 0


def logits_of(T, E, dtype, seed, std=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((T, E), generator=g) * std).to(dtype)


def weight_tolerance(want, logits):
    """exp of a rounded difference (relative error |x| 2^-24, plus one unit of
    expf, 2^-23), a sum of at most 512 such terms over a tree of 21 levels, a
    division, a sum of 32 chosen weights, a division and the scale: each
    factor's relative error adds up."""
    fin = logits[np.isfinite(logits)]
    span = float(fin.max() - fin.min()) if fin.size else 0.0
    return np.abs(want) * (2 * span + 64) * 2.0 ** -24 + 1e-37


CASES = [
    (1, 8, 2, {}), (17, 8, 2, {}), (5, 3, 3, {}), (33, 60, 4, dict(renormalize=False)), (64, 256, 8, dict(scale=2.5)),
    (40, 512, 32, dict(renormalize=False, scale=0.5)), (9, 1, 1, {}),
    (50, 64, 6, dict(score="sigmoid")), (50, 64, 6, dict(score="sigmoid", bias=True, renormalize=False)),
    (70, 256, 8, dict(score="sigmoid", bias=True, n_groups=8, top_groups=4, scale=2.5)),
    (70, 160, 6, dict(bias=True, n_groups=8, top_groups=3, group_best=1, renormalize=False)),
    (41, 60, 4, dict(n_groups=5, top_groups=2)), (30, 96, 5, dict(score="sigmoid", n_groups=32, top_groups=7, group_best=1)),
    (30, 33, 2, dict(score="sigmoid", bias=True, n_groups=11, top_groups=1)), (20, 130, 7, dict(bias=True)),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_route(case, dtype):
    T, E, k, kw = CASES[case]
    kw = dict(kw)
    x = logits_of(T, E, dtype, 100 + case)
    g = torch.Generator().manual_seed(case)
    x[torch.rand((T, E), generator=g) < 0.05] = -INF          # experts that are off
    if T > 4:
        x[1] = -INF                                           # nothing left
        x[2, 1:] = -INF                                       # one expert left
        x[3, 0] = float("nan")
    bias = (torch.rand(E, generator=g) - 0.5) * 0.2 if kw.pop("bias", False) else None
    w, ids = dg.det_moe_route(x.cuda(), k, bias=None if bias is None else bias.cuda(), **kw)
    ok()
    rw, rids = ref.route(ref.f64(x), k, bias=None if bias is None else ref.f64(bias), **kw)
    assert np.array_equal(ids.cpu().numpy(), rids)
    assert (np.abs(ref.f64(w) - rw) <= weight_tolerance(rw, ref.f64(x))).all()


def test_route_ties_go_to_the_lower_index():
    x = torch.zeros(3, 64)
    x[1, 40:] = 1.0
    x[2] = torch.arange(64) // 8
    for kw in ({}, dict(score="sigmoid"), dict(score="sigmoid", bias=torch.zeros(64).cuda()), dict(bias=torch.ones(64).cuda()),
               dict(n_groups=8, top_groups=2), dict(score="sigmoid", n_groups=8, top_groups=2, bias=torch.zeros(64).cuda())):
        _, ids = dg.det_moe_route(x.cuda(), 4, **kw)
        ok()
        b = kw.pop("bias", None)
        _, want = ref.route(ref.f64(x), 4, bias=None if b is None else ref.f64(b), **kw)
        assert np.array_equal(ids.cpu().numpy(), want), kw


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 8])
def test_choices_closer_than_fp32_are_decided_in_64_bits(score, groups):
    """Biases that put many choices within a few FP32 units of each other."""
    T, E = 64, 64
    x = logits_of(T, E, torch.float32, 7)
    s = torch.softmax(x.double(), 1) if score == "softmax" else torch.sigmoid(x.double())
    bias = (0.5 - s[0]).float()                               # row 0: every choice is 0.5 up to rounding
    kw = dict(score=score, n_groups=groups, top_groups=max(1, groups // 2))
    w, ids = dg.det_moe_route(x.cuda(), 8, bias=bias.cuda(), **kw)
    ok()
    _, want = ref.route(ref.f64(x), 8, bias=ref.f64(bias), **kw)
    assert np.array_equal(ids.cpu().numpy(), want)


def test_route_rows_do_not_depend_on_the_batch_or_the_pitch():
    x = logits_of(513, 60, torch.float32, 3).cuda()
    bias = torch.linspace(-0.1, 0.1, 60).cuda()
    kw = dict(score="sigmoid", bias=bias, n_groups=4, top_groups=2)
    w, ids = dg.det_moe_route(x, 5, **kw)
    wide = torch.zeros(513, 77).cuda()
    wide[:, :60] = x
    for rows in (1, 7, 64, 129):
        for src in (x[:rows], wide[:rows, :60], x[100:100 + rows]):
            w2, i2 = dg.det_moe_route(src, 5, **kw)
            lo = 100 if src.data_ptr() == x[100:].data_ptr() else 0
            assert torch.equal(w2.view(torch.int32), w[lo:lo + rows].view(torch.int32)) and torch.equal(i2, ids[lo:lo + rows])
    ok()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_experts_masked_by_the_types_lowest_value(score, dtype):
    """A finite mask: the expert is a candidate, with score 0."""
    x = logits_of(40, 64, dtype, 21)
    g = torch.Generator().manual_seed(2)
    x[torch.rand((40, 64), generator=g) < 0.5] = torch.finfo(dtype).min
    x[3] = torch.finfo(dtype).min
    x[4, 2:] = torch.finfo(dtype).min
    x[5, 1:] = -150.0                                          # scores far below FP32's range next to a large one
    x[5, 7] = -149.0
    bias = (torch.rand(64, generator=g) - 0.5) * 0.2
    for kw in ({}, dict(bias=bias), dict(n_groups=8, top_groups=3), dict(n_groups=8, top_groups=3, bias=bias)):
        b = kw.get("bias")
        w, ids = dg.det_moe_route(x.cuda(), 6, score=score, **dict(kw, bias=None if b is None else b.cuda()))
        ok()
        rw, rids = ref.route(ref.f64(x), 6, score=score, **dict(kw, bias=None if b is None else ref.f64(b)))
        assert np.array_equal(ids.cpu().numpy(), rids), kw
        assert (np.abs(ref.f64(w) - rw) <= np.abs(rw) * (2 * 300 + 64) * 2.0 ** -24 + 1e-37).all()


def test_a_masked_expert_far_away_does_not_move_a_close_choice():
    """Scores 1.5e-8 apart against biases 1e-8 the other way: FP32 cannot tell,
    and an expert that only its bias masks lies beyond the others' range."""
    E, k = 64, 8
    x = (-1e-6 * torch.arange(E, dtype=torch.float64)).float()[None].repeat(3, 1)
    bias = (1e-8 * torch.arange(E, dtype=torch.float64)).float()
    x[:, 40], x[2, 40] = -100.0, -3e38
    bias[40] = -float("inf")
    for kw in ({}, dict(n_groups=8, top_groups=3), dict(n_groups=2, top_groups=1)):
        w, ids = dg.det_moe_route(x.cuda(), k, bias=bias.cuda(), **kw)
        ok()
        rw, rids = ref.route(ref.f64(x), k, bias=ref.f64(bias), **kw)
        assert np.array_equal(ids.cpu().numpy(), rids), kw


@pytest.mark.parametrize("E,groups,top,best", [(64, 8, 3, 2), (512, 32, 5, 1), (12, 6, 2, 2), (30, 2, 1, 2), (256, 8, 4, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_too_close_for_32_bits(E, groups, top, best, score):
    """Rows whose groups hold the same values in other places, shifted by a few
    units of the last place, exact ties among them; with and without a bias."""
    g = torch.Generator().manual_seed(E + groups)
    T, size = 64, E // groups
    base = torch.randn((T, 1, size), generator=g).expand(T, groups, size).clone()
    for t in range(T):
        for h in range(groups):
            base[t, h] = base[t, h, torch.randperm(size, generator=g)]
    x = base.reshape(T, E).contiguous()
    steps = torch.randint(-2, 3, (T, E), generator=g).float() * (torch.arange(T)[:, None] % 3).float()
    x = x + steps * 2.0 ** -23 * x.abs()
    bias = (torch.randint(-2, 3, (E,), generator=g) * 1e-8).float()
    for b in (None, bias):
        kw = dict(n_groups=groups, top_groups=top, group_best=best)
        w, ids = dg.det_moe_route(x.cuda(), 3, score=score, bias=None if b is None else b.cuda(), **kw)
        ok()
        rw, rids = ref.route(ref.f64(x), 3, score=score, bias=None if b is None else ref.f64(b), **kw)
        same = (ids.cpu().numpy() == rids).all(1)
        if b is None:                # values 2^-23 apart or equal: in 64 bits no sum of two lies between
            assert same.all(), np.nonzero(~same)
        else:                        # one step of 1e-8 and 2^-24 apart may lie within 2^-43 of one another
            assert same.mean() >= 0.95, np.nonzero(~same)


def test_route_of_no_tokens():
    w, ids = dg.det_moe_route(torch.zeros(0, 8).cuda(), 2)
    assert w.shape == (0, 2) and ids.shape == (0, 2)
    assert dg.det_moe_route_bwd(w, torch.zeros(0, 8).cuda(), ids).shape == (0, 8)


BWD = [(1, 8, 2, {}), (33, 60, 4, dict(renormalize=False)), (40, 256, 8, dict(scale=2.5)), (50, 64, 6, dict(score="sigmoid")),
       (37, 130, 5, dict(score="sigmoid", renormalize=False, scale=1.5)), (21, 512, 32, dict(renormalize=False))]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", range(len(BWD)))
def test_route_gradient_against_the_formula_and_against_differences(case, dtype):
    T, E, k, kw = BWD[case]
    x = logits_of(T, E, dtype, 200 + case)
    if T > 4:
        x[1] = -INF
        x[2, 2:] = -INF
    g = torch.Generator().manual_seed(case)
    dw = torch.randn((T, k), generator=g)
    _, ids = dg.det_moe_route(x.cuda(), k, **kw)
    got = ref.f64(dg.det_moe_route_bwd(dw.cuda(), x.cuda(), ids, **kw))
    ok()
    score, renorm, scale = kw.get("score", "softmax"), kw.get("renormalize", True), kw.get("scale", 1.0)
    ids = ids.cpu().long()
    want = ref.route_gradient(ref.f64(x), ids.numpy(), ref.f64(dw), score, renorm, scale)
    # Every term is a product of a score (relative error as in the forward
    # test) and (g - sum q g): its size before the cancellation counts.
    live = np.isfinite(ref.f64(x))
    fin = ref.f64(x)[live]
    rel = (4 * float(fin.max() - fin.min()) + 160) * 2.0 ** -24
    gmax = np.abs(ref.f64(dw)).max(1, keepdims=True) * scale
    s = ref.f64(torch.softmax(x.double(), 1)) if score == "softmax" else 1 / (1 + np.exp(-ref.f64(x)))
    s = np.nan_to_num(s)
    chosen = np.zeros((T, E))
    for t in range(T):
        for j in range(k):
            if ids[t, j] >= 0:
                chosen[t, ids[t, j]] = 1
    size = s * 2 * gmax * (1 if not renorm else 1 / np.maximum((s * chosen).sum(1, keepdims=True), 1e-20))
    if renorm or score == "sigmoid":
        size = size * chosen
    half = ref.EPS_F32 if dtype == torch.float32 else ref.EPS_BF16
    assert (np.abs(got - want) <= rel * size + half * np.abs(want) * (1 + rel) + 1e-37).all()
    # Central differences of the weights themselves, in 64 bits.
    t, h = T - 1, 1e-5
    for e in sorted({0, E - 1, int(ids[t, 0])}):
        xp, xm = x.double().clone(), x.double().clone()
        xp[t, e] += h
        xm[t, e] -= h
        f = lambda y: float((ref.weights_of(y, ids, score, renorm, scale) * dw.double()).sum())
        slope = (f(xp) - f(xm)) / (2 * h)
        # truncation h^2 / 6 times a third derivative of at most 6 k |g|, and 1e-13 / h of cancellation
        tol = h * h * k * float(gmax[t, 0]) + 1e-13 * T * k * float(gmax.max()) / h + rel * size[t, e] + 2 * half * abs(slope)
        assert abs(got[t, e] - slope) <= tol, (e, got[t, e], slope)


@pytest.mark.parametrize("T,E,k", [(0, 4, 2), (1, 8, 2), (17, 8, 2), (300, 64, 6), (1000, 512, 3), (1, 1, 1), (4099, 7, 1), (9000, 60, 8)])
def test_dispatch(T, E, k):
    g = torch.Generator().manual_seed(T + E)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    ids[torch.rand((T, k), generator=g) < 0.1] = -1
    if T > 3:
        ids[2] = E + 5                                         # outside: dropped as well
        ids[ids == E // 2] = -1                                # an expert without rows
    off, rows, slots = dg.det_moe_dispatch(ids.cuda(), E)
    ok()
    ro, rr, rs = ref.dispatch(ids.numpy(), E)
    assert np.array_equal(off.cpu().numpy(), ro)
    assert np.array_equal(rows.cpu().numpy(), rr)
    assert np.array_equal(slots.cpu().numpy(), rs)


def test_dispatch_with_every_token_dropped_or_on_one_expert():
    for value in (-1, 3):
        ids = torch.full((777, 2), value, dtype=torch.int32)
        off, rows, slots = dg.det_moe_dispatch(ids.cuda(), 4)
        ok()
        ro, rr, rs = ref.dispatch(ids.numpy(), 4)
        assert np.array_equal(off.cpu().numpy(), ro) and np.array_equal(rows.cpu().numpy(), rr)
        assert np.array_equal(slots.cpu().numpy(), rs)


def rows_of(T, H, seed, std=1.0):
    """BF16 [T, H] inside a wider, 16-byte pitched matrix."""
    g = torch.Generator().manual_seed(seed)
    wide = torch.full((T, (H + 15) // 8 * 8), float("nan"), dtype=torch.bfloat16)
    wide[:, :H] = (torch.randn((T, H), generator=g) * std).bfloat16()
    return wide.cuda()[:, :H]


@pytest.mark.parametrize("T,E,k,H", [(1, 8, 2, 64), (17, 8, 2, 4096), (50, 6, 4, 1000), (33, 4, 1, 7), (300, 16, 6, 129),
                                     (40, 40, 32, 520), (5, 3, 2, 2056)])
def test_gather_combine_and_gradients(T, E, k, H):
    g = torch.Generator().manual_seed(H)
    ids = torch.stack([torch.randperm(max(E, k), generator=g)[:k] for _ in range(T)]).to(torch.int32)
    ids[ids >= E] = -1
    if T > 2:
        ids[1] = -1
    w = torch.rand((T, k), generator=g)
    x, ys, dy, dxs = rows_of(T, H, 1), rows_of(T * k, H, 2), rows_of(T, H, 3), rows_of(T * k, H, 4)
    off, rows, slots = dg.det_moe_dispatch(ids.cuda(), E)
    xs = dg.det_moe_gather(x, rows, k)
    y = dg.det_moe_combine(ys, slots, w.cuda())
    dys, dw = dg.det_moe_combine_bwd(dy, ys, rows, slots, w.cuda())
    dx = dg.det_moe_combine(dxs, slots)
    ok()
    _, rr, rs = ref.dispatch(ids.numpy(), E)
    X, YS, DY, DXS, WW = ref.f64(x), ref.f64(ys), ref.f64(dy), ref.f64(dxs), ref.f64(w)
    want = np.zeros((T * k, H))
    want_dys = np.zeros((T * k, H))
    for r, f in enumerate(rr):
        if f >= 0:
            want[r] = X[f // k]
            want_dys[r] = WW[f // k, f % k] * DY[f // k]
    assert np.array_equal(ref.f64(xs), want)
    # one product in FP32, one rounding to BF16
    assert (np.abs(ref.f64(dys) - want_dys) <= np.abs(want_dys) * (ref.EPS_BF16 + 2.0 ** -23) + 1e-38).all()
    wy, wdx, wdw = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, k))
    sy, sdx, sdw = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            if rs[t, j] >= 0:
                wy[t] += WW[t, j] * YS[rs[t, j]]
                sy[t] += np.abs(WW[t, j] * YS[rs[t, j]])
                wdx[t] += DXS[rs[t, j]]
                sdx[t] += np.abs(DXS[rs[t, j]])
                wdw[t, j] = DY[t] @ YS[rs[t, j]]
                sdw[t, j] = np.abs(DY[t]) @ np.abs(YS[rs[t, j]])
    for got, wnt, size, terms in ((y, wy, sy, k), (dx, wdx, sdx, k)):
        tol = size * terms * 2.0 ** -24
        assert (np.abs(ref.f64(got) - wnt) <= tol + ref.EPS_BF16 * (np.abs(wnt) + tol) + 1e-38).all()
    # a dot product over H: per thread H / 256 terms and 8 columns in a row, then 5 + 8 additions
    assert (np.abs(ref.f64(dw) - wdw) <= sdw * (H // 256 + 8 + 13) * 2.0 ** -24 + 1e-38).all()
    # differences: the combination is linear, so a step in one weight moves it by exactly that row
    if T > 2 and rs[0, 0] >= 0:
        h = 0.5
        wp = WW.copy()
        wp[0, 0] += h
        slope = DY[0] @ ((wp[0, 0] - WW[0, 0]) * YS[rs[0, 0]]) / h
        assert abs(float(dw[0, 0]) - slope) <= sdw[0, 0] * (H // 256 + 21) * 2.0 ** -24 + 1e-9 * sdw[0, 0]


def test_rows_do_not_depend_on_the_batch():
    T, E, k, H = 200, 8, 2, 1032
    g = torch.Generator().manual_seed(0)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32).cuda()
    w = torch.rand((T, k), generator=g).cuda()
    ys_of = rows_of(T * k, H, 5)                                # the row of pair f, wherever it lies
    dy = rows_of(T, H, 6)

    def run(n):
        off, rows, slots = dg.det_moe_dispatch(ids[:n].contiguous(), E)
        ys = ys_of[rows.long()].contiguous()
        y = dg.det_moe_combine(ys, slots, w[:n].contiguous())
        _, dw = dg.det_moe_combine_bwd(dy[:n], ys, rows, slots, w[:n].contiguous())
        return y, dw

    y, dw = run(T)
    for n in (1, 7, 64, 199):
        y2, dw2 = run(n)
        assert torch.equal(y2.view(torch.int16), y[:n].view(torch.int16))
        assert torch.equal(dw2.view(torch.int32), dw[:n].view(torch.int32))
    ok()


def test_on_another_stream():
    s = torch.cuda.Stream()
    x = logits_of(100, 16, torch.float32, 1).cuda()
    w, ids = dg.det_moe_route(x, 2)
    torch.cuda.synchronize()
    w2, ids2 = dg.det_moe_route(x, 2, stream=s)
    off, rows, slots = dg.det_moe_dispatch(ids2, 16, stream=s)
    s.synchronize()
    assert torch.equal(w, w2) and torch.equal(ids, ids2)
    ro, rr, rs = ref.dispatch(ids.cpu().numpy(), 16)
    assert np.array_equal(rows.cpu().numpy(), rr)


def test_the_whole_layer_is_captured_into_a_graph():
    x = logits_of(64, 16, torch.float32, 11).cuda()
    h = rows_of(64, 256, 12)

    def layer():
        w, ids = dg.det_moe_route(x, 2)
        off, rows, slots = dg.det_moe_dispatch(ids, 16)
        xs = dg.det_moe_gather(h, rows, 2)
        return dg.det_moe_combine(xs, slots, w)

    want = layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer()
    x.copy_(logits_of(64, 16, torch.float32, 11).cuda())
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y.view(torch.int16), want.view(torch.int16))
