"""Rows of packed attention that no sequence owns, whatever the bounds around them."""
import pytest
import torch

import attn_ref as ref
import invariant_deterministic_gemm_gb300 as dg
from test_gpu_attn import bounds, make, randn

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def used_memory(*shapes):
    """What new tensors of these shapes are likely to be given: memory that held NaN."""
    for s in shapes:
        torch.full(s, NAN, dtype=torch.bfloat16, device="cuda")


# Rows in front of the first sequence fill whole tiles (of 128 and of 256 rows), and pieces of 512: their queries would see
# keys if they were counted back from a sequence with more keys than queries.
@pytest.mark.parametrize("first", [127, 128, 255, 256, 300, 700, 1000])
@pytest.mark.parametrize("lengths,keys", [((100,), (1000,)), ((1, 0, 60, 3), (700, 5, 900, 3))])
@pytest.mark.parametrize("kw", [dict(), dict(window=90, sinks=5)])
def test_rows_in_front_of_the_first_sequence(first, lengths, keys, kw):
    T, S, H, KV, D = first + sum(lengths) + 9, sum(keys) + 140, 4, 2, 64
    q, _, _ = make(T, 1, H, KV, D, first)
    _, k, v = make(1, S, H, KV, D, first + 1)
    b, kb = bounds(*lengths, start=first), bounds(*keys, start=131)
    dout = randn(5, T, H, D)
    q[:first], dout[:first], q[-9:], dout[-9:] = NAN, INF, INF, NAN
    k[:131], v[:131], k[-9:], v[-9:] = NAN, INF, INF, NAN
    runs = []
    for _ in range(3):
        out = torch.full((T, H, D), NAN, dtype=torch.bfloat16, device="cuda")
        used_memory((H, 2 * T))
        _, lse = dg.det_attn(q, k, v, b, kb, out=out, **kw)
        used_memory((T, H, D), (S, KV, D), (S, KV, D))
        runs.append((out, lse) + dg.det_attn_bwd(dout, q, k, v, out, lse, b, kb, **kw))
    assert dg.det_gemm_check() == 0
    out, lse, dq, dk, dv = runs[0]
    for x in (out, dq):
        assert not x[:first].any() and not x[-9:].any()
    for x in (dk, dv):
        assert not x[:131].any() and not x[-9:].any()
    assert (lse[:, :first] == -INF).all() and (lse[:, -9:] == -INF).all()
    for again in runs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(runs[0], again))
    # the sequences themselves: as without the rows around them
    own, keys_own = slice(first, T - 9), slice(131, S - 9)
    o1, l1 = dg.det_attn(q[own], k[keys_own], v[keys_own], bounds(*lengths), bounds(*keys), **kw)
    g1 = dg.det_attn_bwd(dout[own], q[own], k[keys_own], v[keys_own], o1, l1, bounds(*lengths), bounds(*keys), **kw)
    assert torch.equal(o1, out[own]) and torch.equal(l1, lse[:, own])
    assert torch.equal(g1[0], dq[own]) and torch.equal(g1[1], dk[keys_own]) and torch.equal(g1[2], dv[keys_own])
    want, wl, tol, ltol = ref.attention(q[own], k[keys_own], v[keys_own], bounds(*lengths), bounds(*keys), **kw)
    ref.assert_within(out[own], want, tol, "out")
