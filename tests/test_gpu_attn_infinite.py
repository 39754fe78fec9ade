"""Visible values, keys, queries and gradients that are not finite, whatever their weights and wherever tiles begin."""
import math

import pytest
import torch

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
