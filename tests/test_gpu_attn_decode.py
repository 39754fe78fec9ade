"""Attention of one new token over a paged cache on the GPU against 64 bits."""
import pytest
import torch

import attn_ref as ref
import invariant_deterministic_gemm_gb300 as dg

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32
INF, NAN = float("inf"), float("nan")


def randn(seed, *shape, std=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(BF16).cuda()


def build(lengths, H, KV, D, page, seed=0, heads_first=False, fill=NAN):
    """q, caches, table, lengths, and each sequence's keys and values. All that is no token of a sequence holds `fill`."""
    g = torch.Generator().manual_seed(seed)
    held = [-(-n // page) for n in lengths]
    pages, most = sum(held) + 3, max(held + [1]) + 1
    perm = torch.randperm(pages, generator=g)
    shape = (pages, KV, page, D) if heads_first else (pages, page, KV, D)
    kc, vc = (torch.full(shape, fill, dtype=BF16) for _ in range(2))
    if heads_first:
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    table = torch.full((len(lengths), most), -1, dtype=I32)
    kv, at = [], 0
    for b, n in enumerate(lengths):
        ids = perm[at:at + held[b]]
        at += held[b]
        table[b, :held[b]] = ids.to(I32)
        k, v = (torch.randn((n, KV, D), generator=g).to(BF16) for _ in range(2))
        for j in range(n):
            kc[ids[j // page], j % page], vc[ids[j // page], j % page] = k[j], v[j]
        kv.append((k, v))
    q = (torch.randn((len(lengths), H, D), generator=g) * 1.5).to(BF16)
    move = lambda x: x.transpose(1, 2).cuda().transpose(1, 2) if heads_first else x.cuda()  # noqa: E731
    return q.cuda(), move(kc), move(vc), table.cuda(), torch.tensor(lengths, dtype=I32).cuda(), kv


def check_all(lengths, H, KV, D, page, scale=None, window=None, sinks=0, **kw):
    q, kc, vc, table, n, kv = build(lengths, H, KV, D, page, **kw)
    out = dg.det_attn_decode(q, kc, vc, table, n, scale=scale, window=window, sinks=sinks)
    assert dg.det_gemm_check() == 0
    for b, (k, v) in enumerate(kv):
        want, _, tol, _ = ref.attention(q[b:b + 1], k, v, scale=scale, window=window, sinks=sinks)
        ref.assert_within(out[b:b + 1], want, tol, "sequence %d of %d" % (b, lengths[b]))
    return out


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 127, 128, 129, 255, 256, 257, 511, 513, 1025, 1300])
def test_lengths(n):
    check_all([n], 4, 2, 64, 16, seed=n)


@pytest.mark.parametrize("page", [8, 16, 24, 32, 40, 64, 96, 128, 144, 256])
def test_page_sizes(page):
    check_all([300, 1, 77, 520], 4, 2, 64, page, seed=page)


@pytest.mark.parametrize("D", [8, 16, 40, 64, 72, 96, 120, 128])
def test_head_sizes(D):
    check_all([290, 31], 4, 2, D, 16, seed=D)


@pytest.mark.parametrize("H,KV", [(1, 1), (3, 1), (8, 1), (16, 1), (17, 1), (32, 1), (33, 1), (64, 1), (12, 4), (40, 8), (128, 2), (7, 7)])
def test_shared_heads(H, KV):
    check_all([270, 40, 5], H, KV, 64, 16, seed=H)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (16, 0), (100, 4), (128, 130), (256, 0), (300, 20), (600, 300), (5000, 1)])
def test_windows_and_sinks(window, sinks):
    check_all([1, 90, 256, 700, 1111], 4, 2, 64, 16, window=window, sinks=sinks, seed=window)


def test_ragged_batch_with_empty_sequences():
    out = check_all([0, 400, 0, 1, 33, 0, 260, 128, 0], 8, 2, 128, 32)
    assert not out[0].any() and not out[8].any()


def test_a_cache_with_heads_before_tokens():
    check_all([300, 20], 4, 2, 64, 16, heads_first=True)


@pytest.mark.parametrize("scale", [1e-3, 3.0])
def test_scales(scale):
    check_all([300, 20], 4, 2, 64, 16, scale=scale)


@pytest.mark.parametrize("fill", [INF, -INF, 0.0])
def test_what_lies_behind_a_sequence_does_not_matter(fill):
    a = check_all([300, 20, 129], 4, 2, 64, 16)
    assert torch.equal(a, check_all([300, 20, 129], 4, 2, 64, 16, fill=fill))


def test_hidden_keys_that_are_not_finite():
    """NaN in keys and values that the window hides, in the same tile as seen ones."""
    q, kc, vc, table, n, kv = build([500], 4, 2, 64, 16)
    want = dg.det_attn_decode(q, kc, vc, table, n, window=70, sinks=3)
    for j in list(range(3, 430)):
        kc[table[0, j // 16], j % 16], vc[table[0, j // 16], j % 16] = NAN, INF
    assert torch.equal(dg.det_attn_decode(q, kc, vc, table, n, window=70, sinks=3), want)


def test_values_that_are_not_finite_reach_the_output():
    q, kc, vc, table, n, kv = build([300], 4, 2, 64, 16)
    vc[table[0, 5], 2, 0, 9], vc[table[0, 6], 2, 1, 8] = INF, NAN
    out = dg.det_attn_decode(q, kc, vc, table, n).float()
    assert (out[0, :2, 9] == INF).all() and torch.isnan(out[0, 2:, 8]).all()
    assert int((~torch.isfinite(out)).sum()) == 4


def test_a_sequences_bits_do_not_depend_on_its_batch():
    lengths = [1500, 3, 260, 4100, 1, 777, 2048, 90]
    q, kc, vc, table, n, kv = build(lengths, 16, 2, 128, 16)
    for kw in (dict(), dict(window=600, sinks=4)):
        out = dg.det_attn_decode(q, kc, vc, table, n, **kw)
        for b in range(len(lengths)):
            one = dg.det_attn_decode(q[b:b + 1], kc, vc, table[b:b + 1], n[b:b + 1].clone(), **kw)
            assert torch.equal(one[0], out[b]), (b, kw)
        many = [i % len(lengths) for i in range(301)]
        big = dg.det_attn_decode(q[many], kc, vc, table[many], n[many], **kw)
        assert torch.equal(big, out[many])


def test_many_sequences_and_long_ones():
    """Enough work for every SM several times, beside sequences that are split over all of them."""
    lengths = [20000] + [100 + 7 * i for i in range(200)] + [9000, 0, 1]
    q, kc, vc, table, n, kv = build(lengths, 8, 4, 64, 64)
    out = dg.det_attn_decode(q, kc, vc, table, n)
    assert dg.det_gemm_check() == 0
    for b in (0, 1, 100, 200, 201, 202, 203):
        want, _, tol, _ = ref.attention(q[b:b + 1], *kv[b])
        ref.assert_within(out[b:b + 1], want, tol, "sequence %d" % b)


def test_lengths_and_pages_outside_are_reported():
    q, kc, vc, table, n, kv = build([100, 50, 60], 4, 2, 64, 16, fill=0.0)
    want = dg.det_attn_decode(q, kc, vc, table, n)
    assert dg.det_gemm_check() == 0
    n2 = n.clone()
    n2[1] = -5
    out = dg.det_attn_decode(q, kc, vc, table, n2)
    assert dg.det_gemm_check() == 1
    assert not out[1].any() and torch.equal(out[0], want[0]) and torch.equal(out[2], want[2])
    n2[1] = 1 << 30                                            # counts as all that the table holds, whose last pages are -1
    out = dg.det_attn_decode(q, kc, vc, table, n2)
    assert dg.det_gemm_check() == 1 and torch.isfinite(out.float()).all()
    for bad in (-1, kc.shape[0], 1 << 30):
        t2 = table.clone()
        t2[0, 2] = bad
        out = dg.det_attn_decode(q, kc, vc, t2, n)
        assert dg.det_gemm_check() == 1
        k, v = kv[0]
        keep = [j for j in range(100) if j // 16 != 2]
        w, _, tol, _ = ref.attention(q[:1], k[keep], v[keep])
        ref.assert_within(out[:1], w, tol, "a page outside the cache is hidden")
        assert torch.equal(out[1:], want[1:])


def test_streams_and_two_graphs():
    sets = [build([300, 1000, 5], 8, 2, 64, 16, seed=s)[:5] for s in (1, 2)]
    want = [dg.det_attn_decode(*s) for s in sets]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = dg.det_attn_decode(*sets[0], stream=side)
    side.synchronize()
    assert torch.equal(got, want[0])
    graphs, got = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(dg.det_attn_decode(*s))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # lengths that change between replays, as in a serving loop
    sets[0][4].copy_(torch.tensor([200, 999, 0], dtype=I32))
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], dg.det_attn_decode(*sets[0]))


def test_empty():
    q, kc, vc, table, n, _ = build([10], 4, 2, 64, 16)
    assert dg.det_attn_decode(q[:0], kc, vc, table[:0], n[:0]).shape == (0, 4, 64)
    out = dg.det_attn_decode(q, kc[:0], vc[:0], table[:, :0], torch.zeros_like(n))
    assert not out.any() and dg.det_gemm_check() == 0


def pages_of(lengths, H, KV, D, page, seed):
    """Like build(), for long caches: drawn on the device, every page of the table a page of its own."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    held = [-(-n // page) for n in lengths]
    perm = torch.randperm(sum(held), generator=g, device="cuda").to(I32)
    table = torch.full((len(lengths), max(held)), -1, dtype=I32, device="cuda")
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = perm[at:at + h]
        at += h
    kc, vc = (torch.randn((sum(held), page, KV, D), generator=g, device="cuda", dtype=torch.float32).to(BF16) for _ in range(2))
    q = torch.randn((len(lengths), H, D), generator=g, device="cuda").to(BF16)
    return q, kc, vc, table, torch.tensor(lengths, dtype=I32).cuda()


# Runs of the CTAs that are cut at any chunk, at every fourth, and at every 64th: the work decides, the bits do not tell.
@pytest.mark.parametrize("lengths", [[20000, 700], [45000, 41000, 20000, 1], [20000] + [256] * 80 + [17000]])
@pytest.mark.parametrize("H,KV,D", [(8, 8, 64), (24, 8, 128)])
def test_the_cuts_between_ctas_do_not_show(lengths, H, KV, D):
    q, kc, vc, table, n = pages_of(lengths, H, KV, D, 32, 5)
    out = dg.det_attn_decode(q, kc, vc, table, n)
    assert dg.det_gemm_check() == 0
    for b in (0, 1, len(lengths) - 1):
        one = dg.det_attn_decode(q[b:b + 1], kc, vc, table[b:b + 1], n[b:b + 1].clone())
        assert torch.equal(one[0], out[b])
        ids = table[b, :-(-lengths[b] // 32)].long()
        k, v = (x[ids].flatten(0, 1)[:lengths[b]] for x in (kc, vc))
        want, _, tol, _ = ref.attention(q[b:b + 1], k, v)
        ref.assert_within(out[b:b + 1], want, tol, "sequence %d" % b)


@pytest.mark.parametrize("H,KV", [(1, 1), (3, 3), (15, 5), (40, 1), (64, 1), (35, 7)])
@pytest.mark.parametrize("D", [40, 64, 120])
def test_odd_numbers_of_heads(H, KV, D):
    check_all([700, 0, 33, 1600], H, KV, D, 16)


def test_two_streams_at_once():
    sets = [pages_of([3000, 500, 9000, 1], 16, 4, 128, 16, s) for s in (1, 2)]
    want = [dg.det_attn_decode(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[dg.det_attn_decode(*s, stream=st) for s, st in zip(sets, streams)] for _ in range(8)]
    torch.cuda.synchronize()
    assert dg.det_gemm_check() == 0
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(want, g))


def test_a_timeout_is_reported_and_the_context_stays_usable():
    q, kc, vc, table, n, _ = build([700, 30, 2000], 8, 2, 64, 16)
    want = dg.det_attn_decode(q, kc, vc, table, n)
    assert dg.det_gemm_check() == 0
    dg.det_ops_debug_force_timeout(True)
    try:
        dg.det_attn_decode(q, kc, vc, table, n)
        assert dg.det_gemm_check() == 6
    finally:
        dg.det_ops_debug_force_timeout(False)
    assert torch.equal(dg.det_attn_decode(q, kc, vc, table, n), want)
    assert dg.det_gemm_check() == 0


@pytest.mark.parametrize("order", [(0, 1, 2, 3, 4), (0, 2, 1, 3, 4), (0, 2, 3, 1, 4)])
def test_keys_and_values_in_one_buffer(order):
    """[pages, 2, size, KV, D] with its axes in three orders: appended to and read as two that lie apart."""
    KV, page, D, n = 2, 16, 64, 90
    buffer = torch.zeros([(7, 2, page, KV, D)[i] for i in order], dtype=BF16, device="cuda")
    kv = buffer.permute([order.index(i) for i in range(5)])
    kc, vc = torch.zeros((7, page, KV, D), dtype=BF16, device="cuda"), torch.zeros((7, page, KV, D), dtype=BF16, device="cuda")
    q, k, v = randn(1, n, 4, D), randn(2, n, KV, D), randn(3, n, KV, D)
    angle = torch.randn((n, D // 2), generator=torch.Generator().manual_seed(4)).cuda()
    pos = torch.arange(n, dtype=I32).cuda()
    for a, b in ((kv[:, 0], kv[:, 1]), (kc, vc)):
        dg.det_kv_append(q, k, v, angle.cos(), angle.sin(), pos, pos, a, b)
    assert torch.equal(kv[:, 0], kc) and torch.equal(kv[:, 1], vc)
    table, lengths = torch.arange(6, dtype=I32).cuda()[None], torch.tensor([n], dtype=I32).cuda()
    got = dg.det_attn_decode(q[-1:], kv[:, 0], kv[:, 1], table, lengths)
    assert dg.det_gemm_check() == 0
    assert torch.equal(got, dg.det_attn_decode(q[-1:], kc, vc, table, lengths))
