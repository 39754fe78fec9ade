"""The attention operators at the ends of their ranges: rows whose offsets pass 32 bits, the most heads, thousands of sequences, long
sequences, every head size."""
import pytest
import torch

import attn_ref as ref
import invariant_deterministic_gemm_gb300 as dg
from test_gpu_attn import bounds, make, randn
from test_gpu_rope import tables

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32
NAN = float("nan")


@pytest.fixture
def buffer():
    """A buffer of 2^31 + 2^29 BF16 elements (5.4 GB)."""
    b = torch.empty((1 << 31) + (1 << 29), dtype=BF16, device="cuda")
    yield b
    del b
    torch.cuda.empty_cache()


def far(buffer, shape, strides, offset=0):
    """A view whose last row begins past 2^31 elements (4 GB)."""
    t = torch.as_strided(buffer, shape, strides, offset)
    assert offset + sum((n - 1) * s for n, s in zip(shape, strides)) > 1 << 31
    return t


def test_rotation_and_packed_attention_of_rows_far_apart(buffer):
    T, H, KV, D = 330, 4, 2, 64
    gap = ((1 << 31) // (T - 2) + 512) // 8 * 8
    q, k, v = make(T, T, H, KV, D, 4)
    dout = randn(5, T, H, D)
    places = [far(buffer, (T, n, D), (gap, D, 1), at) for n, at in ((H, 0), (KV, 512), (KV, 1024), (H, 1536))]
    with pytest.raises(dg.DetGemmError, match="overlapping output"):        # (by its first and last byte, though it lies between)
        dg.det_attn(*places[:3], out=far(buffer, (T, H, D), (gap, D, 1), 2048))
    places.append(far(torch.empty_like(buffer), (T, H, D), (gap, D, 1)))
    for x, y in zip(places, (q, k, v, dout)):
        x.copy_(y)
    fq, fk, fv, fd, fo = places
    c, s = tables(T, D)
    pos = torch.arange(T, dtype=I32).cuda()
    assert torch.equal(dg.det_rope(fq, c, s, pos), dg.det_rope(q, c, s, pos))
    assert torch.equal(dg.det_rope(q, c, s, pos, out=fo), dg.det_rope(q, c, s, pos))
    for b, kw in ((None, dict()), (bounds(100, 0, 229, start=1), dict(window=40, sinks=3))):
        out, lse = dg.det_attn(q, k, v, b, **kw)
        o, l = dg.det_attn(fq, fk, fv, b, out=fo, **kw)
        assert torch.equal(o, out) and torch.equal(l, lse)
        for x, y in zip(dg.det_attn_bwd(fd, fq, fk, fv, fo, l, b, **kw), dg.det_attn_bwd(dout, q, k, v, out, lse, b, **kw)):
            assert torch.equal(x, y)
    assert dg.det_gemm_check() == 0


@pytest.mark.parametrize("axis", ["pages", "tokens", "heads"])
def test_a_cache_whose_rows_lie_far_apart(buffer, axis):
    pages, size, KV, D, H, n = 9, 16, 3, 64, 6, 137
    big = {"pages": pages, "tokens": size, "heads": KV}[axis]
    gap = ((1 << 31) // (big - 1) + 4096) // 8 * 8
    strides = {"pages": (gap, KV * D, D, 1), "tokens": (KV * D, gap, D, 1), "heads": (size * D, D, gap, 1)}[axis]
    kc = far(buffer, (pages, size, KV, D), strides)
    vc = far(buffer, (pages, size, KV, D), strides, pages * size * KV * D)
    small = [torch.zeros((pages, size, KV, D), dtype=BF16, device="cuda") for _ in range(2)]
    q, k, v = make(n, n, H, KV, D, 6)
    c, s = tables(n, D)
    pos = torch.arange(n, dtype=I32).cuda()
    table = torch.tensor([[8, 0, 7, 1, 6, 2, 5, 3, 4]], dtype=I32).cuda()
    slots = (table[0].long()[pos.long() // size] * size + pos.long() % size).to(I32)
    got = dg.det_kv_append(q, k, v, c, s, pos, slots, kc, vc)
    want = dg.det_kv_append(q, k, v, c, s, pos, slots, *small)
    assert torch.equal(got, want)
    flat = slots.long()
    for x, y in zip((kc, vc), small):
        assert torch.equal(x[flat // size, flat % size], y[flat // size, flat % size])
    lengths = torch.tensor([n], dtype=I32).cuda()
    for kw in (dict(), dict(window=20, sinks=1)):
        assert torch.equal(dg.det_attn_decode(q[-1:], kc, vc, table, lengths, **kw), dg.det_attn_decode(q[-1:], *small, table, lengths, **kw))
    assert dg.det_gemm_check() == 0


@pytest.mark.parametrize("H,KV", [(1024, 1), (1024, 1024), (1000, 250)])
def test_the_most_heads(H, KV):
    T, D = 37, 16
    q, k, v = make(T, T, H, KV, D, 2)
    dout, b = randn(3, T, H, D), bounds(5, 32)
    out, lse = dg.det_attn(q, k, v, b)
    got = dg.det_attn_bwd(dout, q, k, v, out, lse, b)
    assert dg.det_gemm_check() == 0
    want, wl, tol, ltol = ref.attention(q, k, v, b)
    ref.assert_within(out, want, tol, "out")
    ref.assert_within(lse, wl, ltol, "lse")
    for x, (w, t), n in zip(got, ref.gradients(dout, q, k, v, out, lse, b), ("dq", "dk", "dv")):
        ref.assert_within(x, w, t, n)


@pytest.mark.parametrize("kw", [dict(), dict(window=2, sinks=1)])
def test_thousands_of_short_sequences(kw):
    g = torch.Generator().manual_seed(1)
    lengths = torch.randint(0, 4, (5000,), generator=g).tolist()
    n = sum(lengths)
    q, k, v = make(n, n, 2, 1, 64, 5)
    dout, b = randn(3, n, 2, 64), bounds(*lengths)
    out, lse = dg.det_attn(q, k, v, b, **kw)
    got = dg.det_attn_bwd(dout, q, k, v, out, lse, b, **kw)
    assert dg.det_gemm_check() == 0
    a = int(b[4000])
    for x, y in ((slice(0, int(b[700])), b[:701]), (slice(a, n), b[4000:] - a)):
        y = y.contiguous()
        want, wl, tol, ltol = ref.attention(q[x], k[x], v[x], y, **kw)
        ref.assert_within(out[x], want, tol, "out")
        ref.assert_within(lse[:, x], wl, ltol, "lse")
        for z, (w, t), name in zip(got, ref.gradients(dout[x], q[x], k[x], v[x], out[x], lse[:, x], y, **kw), ("dq", "dk", "dv")):
            ref.assert_within(z[x], w, t, name)


def test_a_long_sequence_with_a_window():
    """The last rows of 150,000, as from a chunk of their own, and the gradients of a loss of theirs."""
    T, last = 150000, 300
    q, k, v = make(T, T, 2, 1, 64, 5)
    kw = dict(window=500, sinks=2)
    out, lse = dg.det_attn(q, k, v, **kw)
    o, l = dg.det_attn(q[-last:], k, v, **kw)
    assert torch.equal(o, out[-last:]) and torch.equal(l, lse[:, -last:])
    dout = torch.zeros_like(out)
    dout[-last:] = randn(3, last, 2, 64)
    full = dg.det_attn_bwd(dout, q, k, v, out, lse, **kw)
    part = dg.det_attn_bwd(dout[-last:], q[-last:], k, v, o, l, **kw)
    assert dg.det_gemm_check() == 0
    assert torch.equal(full[0][-last:], part[0]) and not full[0][:-last].any()
    seen = torch.zeros(T, dtype=torch.bool, device="cuda")
    seen[:2], seen[T - last - 499:] = True, True
    assert not full[1][~seen].any() and not full[2][~seen].any()
    keep = list(range(2)) + list(range(T - last - 499, T))
    i = torch.arange(last)[:, None] + T - last
    j = torch.tensor(keep)[None]
    vis = (j <= i) & ((i - j < 500) | (j < 2))
    for h in range(2):
        s = (ref.f64(q[-last:, h]) @ ref.f64(k[keep, 0]).T / 8).masked_fill(~vis, -float("inf"))
        want = torch.softmax(s, 1) @ ref.f64(v[keep, 0])
        # P and the result rounded to BF16, and FP32's errors of a score of a few units
        off = (torch.softmax(s, 1) @ ref.f64(v[keep, 0]).abs() + want.abs()) * (2.0 ** -8 * 1.01 + 2.0 ** -14)
        ref.assert_within(out[-last:, h], want, off, "out")


@pytest.mark.parametrize("D", range(8, 129, 8))
def test_single_keys_of_every_head_size(D):
    """A query that sees a single key has no dq and gives no dk, in any sum of D products."""
    lengths = (1, 1, 200, 1, 77)
    n = sum(lengths)
    q, k, v = make(n, n, 6, 2, D, D)
    dout, b = randn(9, n, 6, D), bounds(*lengths)
    out, lse = dg.det_attn(q, k, v, b)
    dq, dk, _ = dg.det_attn_bwd(dout, q, k, v, out, lse, b)
    for i in (0, 1, 2, 202, 203):
        assert not dq[i].any()
    for i in (0, 1, 202):
        assert not dk[i].any()
    out, lse = dg.det_attn(q, k, v, b, window=1)
    dq, dk, _ = dg.det_attn_bwd(dout, q, k, v, out, lse, b, window=1)
    assert not dq.any() and not dk.any()
    assert dg.det_gemm_check() == 0
