"""Visible values, keys, queries and gradients that are not finite, whatever their weights and wherever tiles begin."""
import math

import pytest
import torch

import attn_ref as ref
import invariant_deterministic_gemm_gb300 as dg
from test_gpu_attn import bounds, make, randn

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def same(a, b):
    return bool(((a == b) | (torch.isnan(a) & torch.isnan(b))).all())


def with_a_small_weight(T, D, at, KV=2):
    """q, k, v in which key `at` has a weight of zero in FP32 for every query but its own."""
    q, k, v = make(T, T, 2 * KV, KV, D, 3)
    q[:, :, 0], k[at, :, 0] = 8.0, -2000.0
    q[at, :, 0] = 0.0
    return q, k, v


# The chunks' tiles begin at other queries, so that other blocks of keys are seen by all of a tile's rows.
@pytest.mark.parametrize("bad", [INF, -INF, NAN])
@pytest.mark.parametrize("D,kw", [(64, dict()), (128, dict()), (80, dict(window=300, sinks=2))])
def test_an_infinite_value_of_no_weight_in_chunks_of_a_prompt(bad, D, kw):
    T, at = 700, 140
    q, k, v = with_a_small_weight(T, D, at)
    clean, _ = dg.det_attn(q, k, v, **kw)
    v[at, 0, 11] = bad
    out, lse = dg.det_attn(q, k, v, **kw)
    seen = slice(at, at + kw.get("window", T))
    got = out[:, :2, 11].float()
    assert (torch.isnan(got[seen]) if math.isnan(bad) else got[seen] == bad).all()
    rest = torch.ones_like(out, dtype=torch.bool)
    rest[seen, :2, 11] = False
    assert torch.equal(out[rest], clean[rest])
    for cut in (1, 64, 100, 257):
        for a in range(0, T, cut):
            b = min(T, a + cut)
            o, l = dg.det_attn(q[a:b], k[:b], v[:b], **kw)
            assert same(o, out[a:b]) and torch.equal(l, lse[:, a:b]), (cut, a)


def test_infinities_of_both_signs_and_many_of_them():
    T = 1500
    q, k, v = make(T, T, 4, 2, 64, 5)
    v[100, :, 3], v[900, :, 3], v[:, :, 7], v[300:, 1, 9], v[5, :, 12] = INF, -INF, INF, -INF, NAN
    out, _ = dg.det_attn(q, k, v)
    got = out.float()
    assert torch.isfinite(got[:100, :, 3]).all() and (got[100:900, :, 3] == INF).all() and torch.isnan(got[900:, :, 3]).all()
    assert (got[:, :, 7] == INF).all()
    assert (got[300:, 2:, 9] == -INF).all() and torch.isfinite(got[:300, :, 9]).all() and torch.isfinite(got[:, :2, 9]).all()
    assert torch.isfinite(got[:5, :, 12]).all() and torch.isnan(got[5:, :, 12]).all()
    for a, b in ((0, 130), (130, 700), (700, 1500)):
        assert same(dg.det_attn(q[a:b], k[:b], v[:b])[0], out[a:b])


def test_values_of_one_sequence_only():
    """A sequence of infinities and NaN between two others in the same tiles."""
    lengths = (70, 200, 90)
    q, k, v = make(360, 360, 4, 2, 128, 6)
    b = bounds(*lengths)
    clean, _ = dg.det_attn(q, k, v, b)
    v[70:270] = NAN
    v[100:150, :, ::2] = INF
    out, _ = dg.det_attn(q, k, v, b)
    assert torch.equal(out[:70], clean[:70]) and torch.equal(out[270:], clean[270:])
    assert torch.isnan(out[70:270].float()).all()
    assert dg.det_gemm_check() == 0


def gradients(q, k, v, dout, b=None, **kw):
    out, lse = dg.det_attn(q, k, v, b, **kw)
    return [x.float() for x in dg.det_attn_bwd(dout, q, k, v, out, lse, b, **kw)]


@pytest.mark.parametrize("bad", [INF, -INF])
@pytest.mark.parametrize("D,kw", [(64, dict()), (128, dict()), (80, dict(window=300, sinks=2)), (64, dict(window=520, sinks=200))])
def test_infinite_gradients_of_the_output(bad, D, kw):
    """dv of all keys that the query sees, those too to which it gives a weight of zero in FP32, has them with their sign."""
    T, at = 700, 40
    q, k, v = with_a_small_weight(T, D, at)
    for i in (60, 300, 690):                 # their first keys are seen in blocks of queries that are seen in part, and whole
        dout = randn(5, T, 4, D)
        clean = gradients(q, k, v, dout, **kw)
        dout[i, 1, 5] = bad
        dq, dk, dv = gradients(q, k, v, dout, **kw)
        j = torch.arange(T, device="cuda")
        seen = (j <= i) & ((i - j < kw.get("window", T)) | (j < kw.get("sinks", 0)))
        assert (dv[seen, 0, 5] == bad).all(), i
        rest = torch.ones_like(dv, dtype=torch.bool)
        rest[seen, 0, 5] = False
        assert torch.equal(dv[rest], clean[2][rest]), i
        assert torch.equal(dk[:, 1], clean[1][:, 1]) and torch.equal(dk[~seen], clean[1][~seen]), i
        others = torch.arange(T, device="cuda") != i
        assert torch.equal(dq[others], clean[0][others]), i


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("D,kw", [(64, dict()), (128, dict()), (80, dict(window=300, sinks=2))])
def test_keys_and_queries_with_scores_of_minus_infinity(sign, D, kw):
    """Their P and dS are zero, and zero times infinity is NaN: in that column of dq, for the queries that see the key, and of dk,
    for the keys that the query sees, in whichever block."""
    T, at = 700, 140
    q, k, v = make(T, T, 4, 2, D, 7)
    dout, j = randn(5, T, 4, D), torch.arange(T, device="cuda")
    window, sinks = kw.get("window", T), kw.get("sinks", 0)
    q[:, :, 3], k[:, :, 3] = sign, 0.0
    clean = gradients(q, k, v, dout, **kw)
    k[at, 1, 3] = -sign * INF
    got = gradients(q, k, v, dout, **kw)
    sees = (j >= at) & (j - at < window)
    assert torch.isnan(got[0][sees][:, 2:, 3]).all()
    assert torch.isfinite(got[0][~sees]).all() and torch.isfinite(got[0][:, :2]).all() and torch.isfinite(got[0][..., :3]).all()
    assert torch.equal(got[0][:, :2], clean[0][:, :2]) and torch.equal(got[0][:at], clean[0][:at])
    # a query whose scores are all -infinity
    q, k, v = make(T, T, 4, 2, D, 7)
    k[:, :, 3] = -sign
    clean = gradients(q, k, v, dout, **kw)
    q[at, 2, 3] = sign * INF
    got = gradients(q, k, v, dout, **kw)
    seen = (j <= at) & ((at - j < window) | (j < sinks))
    assert torch.isnan(got[1][seen][:, 1, 3]).all()
    assert torch.equal(got[1][~seen], clean[1][~seen]) and torch.equal(got[1][:, 0], clean[1][:, 0])
    assert torch.isfinite(got[1][:, 1, 4:]).all() and torch.isfinite(got[2]).all()


def test_gradients_of_a_sequence_between_others():
    lengths = (70, 200, 90)
    q, k, v = make(360, 360, 4, 2, 128, 6)
    b, dout = bounds(*lengths), randn(8, 360, 4, 128)
    clean = gradients(q, k, v, dout, b)
    for x in (q, k, v, dout):
        x[70:270] = NAN
        x[100:150, :, ::2] = INF
    got = gradients(q, k, v, dout, b)
    for x, y in zip(got, clean):
        assert torch.equal(x[:70], y[:70]) and torch.equal(x[270:], y[270:]) and torch.isnan(x[71:270]).all()
    assert dg.det_gemm_check() == 0


@pytest.mark.parametrize("D", [64, 128])
def test_scores_of_minus_infinity_alone_give_zeros(D):
    """In packed attention and in the decode, as if no key were seen; beside a finite score they weigh nothing."""
    T, page = 200, 16
    q, k, v = make(T, T, 4, 2, D, 4)
    q[:, :, 3], k[:150, :, 3], k[150:, :, 3] = 1.0, -INF, 0.0
    out, lse = dg.det_attn(q, k, v)
    assert not out[:150].any() and (lse[:, :150] == -INF).all()
    want, wl, tol, ltol = ref.attention(q[150:], k[150:], v[150:])
    ref.assert_within(out[150:], want, tol, "out")
    ref.assert_within(lse[:, 150:], wl, ltol, "lse")
    pages = -(-T // page)
    kc, vc = (torch.zeros((pages, page, 2, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kc.view(-1, 2, D)[:T], vc.view(-1, 2, D)[:T] = k, v
    table = torch.arange(pages, dtype=torch.int32).cuda()[None].expand(3, -1).contiguous()
    n = torch.tensor([1, 150, T], dtype=torch.int32).cuda()
    got = dg.det_attn_decode(q[[0, 149, T - 1]], kc, vc, table, n)
    assert not got[:2].any()
    ref.assert_within(got[2], want[-1], tol[-1], "decode")
    # an infinite value of no weight: multiplied with it in the decode
    vc[0, 0, 0, 5] = INF
    got = dg.det_attn_decode(q[[T - 1] * 3], kc, vc, table, n)
    assert torch.isnan(got[2, :2, 5]).all() and int((~torch.isfinite(got[2])).sum()) == 2
    assert dg.det_gemm_check() == 0
