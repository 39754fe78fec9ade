"""Attention of packed sequences and its gradients on the GPU against 64 bits:
head sizes, shared heads, windows and sinks, ragged and empty sequences, what
masked places hold, and the same bits in any batch and cut."""
import math

import pytest
import torch

import attn_ref as ref
import invariant_deterministic_gemm_gb300 as dg

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32
INF, NAN = float("inf"), float("nan")


def randn(seed, *shape, std=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(BF16).cuda()


def make(T, S, H, KV, D, seed=0):
    """q, k, v as views of one buffer each, with strides of their own."""
    q = randn(seed, T, H + 2, D, std=1.5)[:, 1:H + 1]
    kv = randn(seed + 1, S, 2 * KV, D)
    return q, kv[:, :KV], kv[:, KV:]


def bounds(*lengths, start=0):
    b = [start]
    for n in lengths:
        b.append(b[-1] + n)
    return torch.tensor(b, dtype=I32).cuda()


def check_all(q, k, v, b=None, kb=None, grads=True, **kw):
    out, lse = dg.det_attn(q, k, v, b, kb, **kw)
    assert dg.det_gemm_check() == 0
    want, wl, tol, ltol = ref.attention(q, k, v, b, kb, **kw)
    ref.assert_within(out, want, tol, "out")
    got, inf = ref.f64(lse), torch.isinf(wl)
    assert torch.equal(got[inf], wl[inf])
    ref.assert_within(got[~inf], wl[~inf], ltol[~inf], "lse")
    if not grads:
        return out, lse
    dout = randn(77, *q.shape, std=1e-2)
    got = dg.det_attn_bwd(dout, q, k, v, out, lse, b, kb, **kw)
    assert dg.det_gemm_check() == 0
    for name, x, (w, t) in zip(("dq", "dk", "dv"), got, ref.gradients(dout, q, k, v, out, lse, b, kb, **kw)):
        ref.assert_within(x, w, t, name)
    return (out, lse) + tuple(got)


@pytest.mark.parametrize("T", [1, 2, 31, 127, 128, 129, 255, 257, 400])
def test_lengths(T):
    check_all(*make(T, T, 2, 1, 64, T))


@pytest.mark.parametrize("D", [8, 16, 24, 40, 64, 72, 80, 96, 120, 128])
def test_head_sizes(D):
    check_all(*make(200, 200, 2, 2, D, D))


@pytest.mark.parametrize("H,KV", [(1, 1), (3, 1), (8, 2), (6, 6), (5, 5), (14, 2)])
def test_shared_heads(H, KV):
    check_all(*make(150, 150, H, KV, 48, H))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (2, 1), (17, 0), (100, 4), (128, 0), (129, 130), (200, 1), (256, 300), (5000, 2)])
def test_windows_and_sinks(window, sinks):
    check_all(*make(420, 420, 2, 1, 64, window), window=window, sinks=sinks)


@pytest.mark.parametrize("lengths", [(1,), (1, 1, 1), (0, 5, 0, 0, 130, 1, 0), (128, 128), (127, 129, 3), (300, 0, 200), (256, 256, 1)])
@pytest.mark.parametrize("window", [None, 60])
def test_packed_sequences(lengths, window):
    n = sum(lengths)
    check_all(*make(n, n, 4, 2, 64, n), bounds(*lengths), window=window, sinks=2)


@pytest.mark.parametrize("lengths", [(5, 0, 130, 1), (64,)])
def test_rows_outside_the_sequences_are_zeros(lengths):
    n = sum(lengths) + 20
    q, k, v = make(n, n, 2, 1, 64, 5)
    q[:7], k[:7], v[:7], q[-13:], k[-13:], v[-13:] = NAN, INF, NAN, INF, NAN, INF
    r = check_all(q, k, v, bounds(*lengths, start=7))
    for x in (r[0],) + r[2:]:
        assert not x[:7].any() and not x[-13:].any()
    assert (r[1][:, :7] == -INF).all()


@pytest.mark.parametrize("nq,nk", [((1, 1, 1), (1, 200, 513)), ((5, 0, 100), (5, 30, 400)), ((128, 300), (257, 300)), ((10, 40), (3, 40)),
                                   ((200,), (0,)), ((0, 3), (50, 130)), ((150,), (20,))])
@pytest.mark.parametrize("window", [None, 33])
def test_chunks_of_queries(nq, nk, window):
    """Fewer queries than keys, as in a prompt's later chunks; more queries than keys leaves rows that see nothing."""
    q, _, _ = make(sum(nq), 1, 4, 2, 64, 3)
    _, k, v = make(1, sum(nk), 4, 2, 64, 4)
    check_all(q, k, v, bounds(*nq), bounds(*nk), window=window, sinks=3)


def test_one_sequence_without_bounds_may_have_more_keys():
    q, _, _ = make(40, 1, 2, 1, 64, 3)
    _, k, v = make(1, 333, 2, 1, 64, 4)
    check_all(q, k, v)


@pytest.mark.parametrize("scale", [1e-3, 0.125, 4.0])
def test_scales(scale):
    check_all(*make(260, 260, 2, 1, 64, 8), scale=scale)


def test_scores_that_rise_and_fall_along_the_keys():
    """Maxima that grow block by block, and one early key that keeps the maximum."""
    q, k, v = make(700, 700, 2, 1, 64, 8)
    k.mul_(torch.linspace(0.1, 12.0, 700, device="cuda")[:, None, None])
    check_all(q, k, v)
    k.copy_(k.flip(0))
    check_all(q, k, v)


@pytest.mark.parametrize("window", [None, 50])
@pytest.mark.parametrize("bad", [INF, -INF, NAN])
def test_later_tokens_do_not_reach_earlier_rows(bad, window):
    """Infinities and NaN in keys, values, queries and gradients of later tokens, of the same tile too."""
    T, cut = 300, 130
    q, k, v = make(T, T, 4, 2, 64, 9)
    dout = randn(5, T, 4, 64)
    kw = dict(window=window, sinks=1)
    a = dg.det_attn(q[:cut], k[:cut], v[:cut], **kw)
    k[cut:, :, 5], v[cut:, :, 7], q[cut:, :, 3] = bad, bad, bad
    b = dg.det_attn(q, k, v, **kw)
    assert torch.equal(a[0], b[0][:cut]) and torch.equal(a[1], b[1][:, :cut])
    ga = dg.det_attn_bwd(dout[:cut], q[:cut], k[:cut], v[:cut], *a, **kw)[0]
    gb = dg.det_attn_bwd(dout, q, k, v, *b, **kw)[0]
    assert torch.equal(ga, gb[:cut])
    assert dg.det_gemm_check() == 0


@pytest.mark.parametrize("bad", [INF, -INF, NAN])
def test_values_that_are_not_finite_reach_the_rows_that_see_them(bad):
    T, at = 260, 140
    q, k, v = make(T, T, 2, 1, 64, 10)
    v[at, 0, 11] = bad
    out, _ = dg.det_attn(q, k, v)
    got = out[:, :, 11].float()
    assert torch.isfinite(got[:at]).all()
    assert torch.isnan(got[at:]).all() if math.isnan(bad) else (got[at:] == bad).all()
    rest = torch.cat([out[..., :11], out[..., 12:]], -1)
    assert torch.isfinite(rest.float()).all()


@pytest.mark.parametrize("bad", [INF, NAN])
def test_gradients_of_other_sequences_do_not_mix(bad):
    """A sequence whose gradient overflowed, beside others in the same tiles."""
    q, k, v = make(200, 200, 4, 2, 64, 11)
    b, dout = bounds(60, 45, 95), randn(5, 200, 4, 64)
    out, lse = dg.det_attn(q, k, v, b)
    want = dg.det_attn_bwd(dout, q, k, v, out, lse, b)
    dout[60:105, :, 3] = bad
    got = dg.det_attn_bwd(dout, q, k, v, out, lse, b)
    for x, y in zip(want, got):
        assert torch.equal(x[:60], y[:60]) and torch.equal(x[105:], y[105:])
        assert not torch.isfinite(y[60:105].float()).all()


@pytest.mark.parametrize("kw", [dict(), dict(window=70, sinks=2)])
def test_a_sequences_bits_do_not_depend_on_its_batch(kw):
    lengths = (1, 130, 77, 500, 256)
    n = sum(lengths)
    q, k, v = make(n, n, 4, 2, 80, 12)
    dout, b = randn(6, n, 4, 80), bounds(*lengths)
    out, lse = dg.det_attn(q, k, v, b, **kw)
    g = dg.det_attn_bwd(dout, q, k, v, out, lse, b, **kw)
    for again in range(2):
        o2, l2 = dg.det_attn(q, k, v, b, **kw)
        g2 = dg.det_attn_bwd(dout, q, k, v, o2, l2, b, **kw)
        assert torch.equal(out, o2) and torch.equal(lse, l2) and all(torch.equal(x, y) for x, y in zip(g, g2))
    a = 0
    for m in lengths:
        s = slice(a, a + m)
        o1, l1 = dg.det_attn(q[s], k[s], v[s], **kw)
        g1 = dg.det_attn_bwd(dout[s], q[s], k[s], v[s], o1, l1, **kw)
        assert torch.equal(out[s], o1) and torch.equal(lse[:, s], l1)
        assert all(torch.equal(x[s], y) for x, y in zip(g, g1))
        a += m


@pytest.mark.parametrize("kw", [dict(), dict(window=90, sinks=5)])
def test_a_prompts_bits_do_not_depend_on_its_chunks(kw):
    T = 700
    q, k, v = make(T, T, 4, 2, 128, 13)
    out, lse = dg.det_attn(q, k, v, **kw)
    for cut in (1, 64, 100, 257):
        for a in range(0, T, cut):
            b = min(T, a + cut)
            o, l = dg.det_attn(q[a:b], k[:b], v[:b], **kw)
            assert torch.equal(out[a:b], o) and torch.equal(lse[:, a:b], l), (cut, a)


def test_gradients_against_differences():
    """The loss sum(out * w) along random directions: (f(x + h) - f(x - h)) / 2h in 64 bits, and the gradient's
    product with the direction, within the gradient's own bounds."""
    T, H, KV, D = 90, 4, 2, 32
    q, k, v = make(T, T, H, KV, D, 14)
    w, b, kw = randn(3, T, H, D), bounds(40, 50), dict(window=25, sinks=2)
    out, lse = dg.det_attn(q, k, v, b, **kw)
    got = dg.det_attn_bwd(w, q, k, v, out, lse, b, **kw)
    exact = ref.gradients(w, q, k, v, out, lse, b, **kw)
    x = [ref.f64(t) for t in (q, k, v)]
    for i in range(3):
        d = torch.randn(x[i].shape, generator=torch.Generator().manual_seed(i), dtype=ref.F64)
        f = []
        for h in (1e-4, -1e-4):
            y = list(x)
            y[i] = x[i] + h * d
            f.append(float((ref.attention(*y, b, **kw)[0] * ref.f64(w)).sum()))
        want = (f[0] - f[1]) / 2e-4
        # besides the gradient's bounds: delta comes from out rounded to BF16, a part of scale |delta| U16 sum |p k| of dq
        off = float((exact[i][1] * d.abs()).sum()) + 0.01 * float((exact[i][0].abs() * d.abs()).sum())
        assert abs(float((ref.f64(got[i]) * d).sum()) - want) <= off, i


def test_streams_and_a_given_output():
    q, k, v = make(300, 300, 4, 2, 64, 15)
    want = dg.det_attn(q, k, v)
    torch.cuda.synchronize()
    side, buf = torch.cuda.Stream(), torch.zeros(300, 9, 64, dtype=BF16, device="cuda")
    torch.cuda.synchronize()
    out, lse = dg.det_attn(q, k, v, out=buf[:, 2:6], stream=side)
    side.synchronize()
    assert out.data_ptr() == buf[:, 2:6].data_ptr() and torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert not buf[:, :2].any() and not buf[:, 6:].any()


def test_two_graphs_replayed_in_turn():
    """Forward and backward captured twice on different inputs, while eager results of the same tensors live."""
    sets = [make(270, 270, 4, 2, 64, s) + (randn(s, 270, 4, 64),) for s in (20, 30)]

    def step(q, k, v, d):
        out, lse = dg.det_attn(q, k, v, window=100, sinks=2)
        return (out, lse) + dg.det_attn_bwd(d, q, k, v, out, lse, window=100, sinks=2)

    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    graphs, got = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(step(*s))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_bounds_that_leave_the_rows_or_go_down_are_reported():
    q, k, v = make(50, 50, 2, 1, 64, 16)
    for b in ([0, 60], [-3, 50], [0, 30, 20, 50], [10, 5]):
        t = torch.tensor(b, dtype=I32).cuda()
        out, lse = dg.det_attn(q, k, v, t)
        assert dg.det_gemm_check() == 1, b
        dg.det_attn_bwd(q, q, k, v, out, lse, t)
        assert dg.det_gemm_check() in (0, 1)
    dg.det_attn(q, k, v, bounds(50))
    assert dg.det_gemm_check() == 0


def test_empty_calls():
    q, k, v = make(0, 0, 2, 1, 64)
    out, lse = dg.det_attn(q, k, v)
    assert out.shape == (0, 2, 64) and lse.shape == (2, 0)
    assert [x.shape[0] for x in dg.det_attn_bwd(out, q, k, v, out, lse)] == [0, 0, 0]
    q, _, _ = make(5, 1, 2, 1, 64)
    out, lse = dg.det_attn(q, k, v)
    assert not out.any() and (lse == -INF).all()
    assert not dg.det_attn_bwd(out, q, k, v, out, lse)[0].any()
    k, v = randn(1, 6, 1, 64), randn(2, 6, 1, 64)
    q0 = q[:0]
    out, lse = dg.det_attn(q0, k, v)
    _, dk, dv = dg.det_attn_bwd(out, q0, k, v, out, lse)
    assert not dk.any() and not dv.any()
    none = torch.zeros(1, dtype=I32).cuda()
    out, lse = dg.det_attn(q, k[:5], v[:5], none)                      # no sequences: rows of nobody
    assert not out.any() and (lse == -INF).all()
    assert dg.det_gemm_check() == 0


# The first keys' gradients are those of every query, in pieces of 512 queries (of up to 512 such keys); beyond that in one.
@pytest.mark.parametrize("sinks,window,lengths", [(5, 200, (1300, 700)), (130, 100, (1100,)), (600, 64, (1000, 3, 530)), (512, 1, (1025,))])
def test_first_keys_over_several_pieces_of_queries(sinks, window, lengths):
    n = sum(lengths)
    q, k, v = make(n, n, 4, 2, 64, 31)
    check_all(q, k, v, bounds(*lengths), window=window, sinks=sinks)


def test_first_keys_of_chunks_of_queries():
    q, k, v = make(1200, 2100, 2, 1, 72, 32)
    check_all(q, k, v, bounds(700, 500), bounds(900, 1200), window=90, sinks=5)


@pytest.mark.parametrize("kw", [dict(window=70, sinks=140), dict()])
def test_the_bits_of_long_sequences_do_not_depend_on_their_batch(kw):
    lengths = (1300, 40, 1030)
    n = sum(lengths)
    q, k, v = make(n, n, 4, 2, 128, 33)
    dout, b = randn(8, n, 4, 128), bounds(*lengths)
    out, lse = dg.det_attn(q, k, v, b, **kw)
    g = dg.det_attn_bwd(dout, q, k, v, out, lse, b, **kw)
    a = 0
    for m in lengths:
        s = slice(a, a + m)
        o1, l1 = dg.det_attn(q[s], k[s], v[s], **kw)
        g1 = dg.det_attn_bwd(dout[s], q[s], k[s], v[s], o1, l1, **kw)
        assert torch.equal(out[s], o1) and torch.equal(lse[:, s], l1)
        assert all(torch.equal(x[s], y) for x, y in zip(g, g1))
        a += m


@pytest.mark.parametrize("kw", [dict(), dict(window=200, sinks=3)])
def test_steps_behind_one_another(kw):
    """Launches that begin while the ones in front end, caches warm: the same bits every time."""
    sets = [make(900, 900, 8, 2, 128, s) + (randn(s, 900, 8, 128),) for s in (61, 62)]

    def step(x):
        q, k, v, dout = x
        out, lse = dg.det_attn(q, k, v, **kw)
        return (out, lse) + dg.det_attn_bwd(dout, q, k, v, out, lse, **kw)

    want = []
    for x in sets:
        want.append(step(x))
        torch.cuda.synchronize()
    for _ in range(10):
        got = [step(sets[i & 1]) for i in range(20)]
        torch.cuda.synchronize()
        for i, one in enumerate(got):
            assert all(torch.equal(x, y) for x, y in zip(want[i & 1], one))


def test_two_streams_at_once():
    sets = [make(900, 900, 8, 2, 128, s) + (randn(s, 900, 8, 128),) for s in (41, 42)]
    kw = dict(window=200, sinks=3)

    def step(x, stream=None):
        q, k, v, dout = x
        out, lse = dg.det_attn(q, k, v, stream=stream, **kw)
        return (out, lse) + dg.det_attn_bwd(dout, q, k, v, out, lse, stream=stream, **kw)

    want = [step(x) for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            got[i].append(step(sets[i], s))
    torch.cuda.synchronize()
    assert dg.det_gemm_check() == 0
    for w, g in zip(want, got):
        for one in g:
            assert all(torch.equal(x, y) for x, y in zip(w, one))


def test_a_timeout_is_reported_and_the_context_stays_usable():
    q, k, v = make(300, 300, 4, 2, 64, 51)
    dout = randn(52, 300, 4, 64)
    kw = dict(window=50, sinks=2)
    out, lse = dg.det_attn(q, k, v, **kw)
    g = dg.det_attn_bwd(dout, q, k, v, out, lse, **kw)
    assert dg.det_gemm_check() == 0
    dg.det_ops_debug_force_timeout(True)
    try:
        dg.det_attn(q, k, v, **kw)
        assert dg.det_gemm_check() == 6
        dg.det_attn_bwd(dout, q, k, v, out, lse, **kw)
        assert dg.det_gemm_check() == 6
    finally:
        dg.det_ops_debug_force_timeout(False)
    o2, l2 = dg.det_attn(q, k, v, **kw)
    g2 = dg.det_attn_bwd(dout, q, k, v, o2, l2, **kw)
    assert dg.det_gemm_check() == 0
    assert torch.equal(out, o2) and torch.equal(lse, l2) and all(torch.equal(x, y) for x, y in zip(g, g2))


@pytest.mark.parametrize("lengths,kw", [((1, 1, 1), {}), ((1,), {}), ((300, 1, 70), dict(window=1))])
def test_queries_that_see_a_single_key_have_no_gradient(lengths, kw):
    n = sum(lengths)
    q, k, v = make(n, n, 6, 2, 72, 71)
    dout, b = randn(9, n, 6, 72), bounds(*lengths)
    out, lse = dg.det_attn(q, k, v, b, **kw)
    assert torch.equal(out, v.repeat_interleave(3, 1))
    dq, dk, dv = dg.det_attn_bwd(dout, q, k, v, out, lse, b, **kw)
    assert dg.det_gemm_check() == 0
    assert not dq.any() and not dk.any()
    want = ref.f64(dout).unflatten(1, (2, 3)).sum(2)
    ref.assert_within(dv, want, ref.f64(dout).abs().unflatten(1, (2, 3)).sum(2) * (2.0 ** -8 + 2.0 ** -20), "dv")


def test_the_first_query_of_a_sequence_has_no_gradient():
    q, k, v = make(400, 400, 4, 2, 128, 72)
    b = bounds(200, 200)
    out, lse = dg.det_attn(q, k, v, b)
    dout = torch.zeros_like(out)
    dout[0], dout[200] = randn(1, 4, 128), randn(2, 4, 128)
    dq, dk, dv = dg.det_attn_bwd(dout, q, k, v, out, lse, b)
    assert not dq.any() and not dk.any() and dv[0].any() and dv[200].any()
