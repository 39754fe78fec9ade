"""Gradients of a range of keys, from the out and lse of more keys than these (results over several ranges, joined)."""
import pytest
import torch

import attn_ref as ref
import invariant_deterministic_gemm_gb300 as dg
from test_gpu_attn import bounds, make, randn

pytestmark = pytest.mark.gpu
NAMES = ("dq", "dk", "dv")


def assert_gradients(got, dout, q, k, v, out, lse, *b, **kw):
    assert dg.det_gemm_check() == 0
    for name, x, (w, t) in zip(NAMES, got, ref.gradients(dout, q, k, v, out, lse, *b, **kw)):
        ref.assert_within(x, w, t, name)


@pytest.mark.parametrize("D", [64, 80, 128])
@pytest.mark.parametrize("T,before", [(1, 1), (1, 200), (130, 1), (200, 300)])
def test_a_causal_range_of_a_sequence(T, before, D):
    """The first query sees one of these keys, with less than all of its weight."""
    q, _, _ = make(T, 1, 4, 2, D, T)
    _, k, v = make(1, before + T, 4, 2, D, D)
    dout = randn(9, T, 4, D)
    out, lse = dg.det_attn(q, k, v)
    k1, v1 = k[before:], v[before:]
    got = dg.det_attn_bwd(dout, q, k1, v1, out, lse)
    assert_gradients(got, dout, q, k1, v1, out, lse)
    assert got[0][0].any() and got[1][0].any()
    # both ranges' gradients together are the whole's (each rounded once to BF16, and dq's sum of two)
    whole = dg.det_attn_bwd(dout, q, k, v, out, lse)
    k0, v0 = k[:before], v[:before]
    s = torch.einsum("thd,shd->hts", ref.f64(q), ref.f64(k0).repeat_interleave(2, 1)) * D ** -0.5
    p = torch.exp(s - ref.f64(lse)[:, :, None])
    dp = torch.einsum("thd,shd->hts", ref.f64(dout), ref.f64(v0).repeat_interleave(2, 1))
    ds = p * (dp - (ref.f64(dout) * ref.f64(out)).sum(2).T[:, :, None])
    dq0 = torch.einsum("hts,shd->thd", ds, ref.f64(k0).repeat_interleave(2, 1)) * D ** -0.5
    _, tol = ref.gradients(dout, q, k, v, out, lse)[0]
    ref.assert_within(whole[0], ref.f64(got[0]) + dq0, tol + ref.gradients(dout, q, k1, v1, out, lse)[0][1], "dq of both ranges")


def test_packed_ranges_and_heads():
    """Several sequences, shared heads: some lse over more keys, some their own."""
    lengths, T = (1, 130, 1, 70), 202
    q, k, v = make(T, T, 6, 2, 72, 3)
    b, dout = bounds(*lengths), randn(4, T, 6, 72)
    out, lse = dg.det_attn(q, k, v, b)
    own = dg.det_attn_bwd(dout, q, k, v, out, lse, b)
    for a in (0, 1, 131, 132):
        assert not own[0][a].any()
    # the second and third sequence's rows as if half of each sum lay elsewhere, with other values there
    lse2, out2 = lse.clone(), out.clone()
    lse2[:, 1:132] += 0.6931471805599453
    out2[1:132] = ((out[1:132].float() + randn(5, 131, 6, 72).float()) / 2).to(out.dtype)
    got = dg.det_attn_bwd(dout, q, k, v, out2, lse2, b)
    assert_gradients(got, dout, q, k, v, out2, lse2, b)
    assert got[0][1].any() and got[0][131].any() and got[1][131].any()
    assert not got[0][0].any() and not got[0][132].any()


@pytest.mark.parametrize("lengths", [(300,), (129, 1, 40)])
def test_a_window_of_one(lengths):
    """Every query sees one key of these, itself: of its own lse nothing, of a larger one the formula's."""
    T = sum(lengths)
    q, k, v = make(T, T, 4, 2, 64, 8)
    b, dout = bounds(*lengths), randn(6, T, 4, 64)
    out, lse = dg.det_attn(q, k, v, b, window=1)
    got = dg.det_attn_bwd(dout, q, k, v, out, lse, b, window=1)
    assert not got[0].any() and not got[1].any()
    lse2 = lse + torch.rand(lse.shape, generator=torch.Generator().manual_seed(1)).cuda()
    got = dg.det_attn_bwd(dout, q, k, v, out, lse2, b, window=1)
    assert_gradients(got, dout, q, k, v, out, lse2, b, window=1)


@pytest.mark.parametrize("scale", [1e-3, 1.0, 30.0])
def test_single_keys_with_large_scores(scale):
    """The weight of a single key is one to within FP32's error of its score, small or large."""
    q, k, v = make(140, 140, 4, 2, 128, 9)
    b, dout = bounds(1, 1, 138), randn(7, 140, 4, 128)
    out, lse = dg.det_attn(q, k, v, b, scale=scale)
    dq, dk, _ = dg.det_attn_bwd(dout, q, k, v, out, lse, b, scale=scale)
    assert not dq[:3].any() and not dk[:2].any()
