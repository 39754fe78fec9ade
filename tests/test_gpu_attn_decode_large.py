"""Batches of more sequences than a block of the decode has threads: its look at the lengths goes round more than once."""
import pytest
import torch

import attn_ref as ref
import invariant_deterministic_gemm_gb300 as dg
from test_gpu_attn_decode import pages_of

pytestmark = pytest.mark.gpu
I32 = torch.int32


def lengths_of(B, kind):
    g = torch.Generator().manual_seed(B)
    if kind == "ragged":
        n = torch.randint(0, 400, (B,), generator=g)
        n[torch.rand(B, generator=g) < 0.3] = 0
        n[7], n[B - 2], n[B - 1] = 3000, 1, 2100
    elif kind == "last alone":
        n = torch.zeros(B, dtype=torch.int64)
        n[B - 1] = 900
    else:
        n = torch.ones(B, dtype=torch.int64)
    return n.tolist()


@pytest.mark.parametrize("B", [511, 512, 513, 1024, 1025, 1700])
@pytest.mark.parametrize("kind", ["ragged", "last alone", "ones"])
@pytest.mark.parametrize("H,KV,D,kw", [(8, 2, 64, dict()), (6, 6, 128, dict(window=100, sinks=3))])
def test_more_sequences_than_threads(B, kind, H, KV, D, kw):
    lengths = lengths_of(B, kind)
    q, kc, vc, table, n = pages_of(lengths, H, KV, D, 16, B)
    out = dg.det_attn_decode(q, kc, vc, table, n, **kw)
    assert dg.det_gemm_check() == 0
    empty = torch.tensor([x == 0 for x in lengths], device="cuda")
    assert not out[empty].any()
    if kind == "ones":
        assert torch.equal(out, vc[table[:, 0].long(), 0].repeat_interleave(H // KV, 1))
    for b in sorted({0, 7, 510, min(511, B - 1), B // 2, min(512, B - 1), min(1024, B - 1), B - 2, B - 1}):
        one = dg.det_attn_decode(q[b:b + 1], kc, vc, table[b:b + 1], n[b:b + 1].clone(), **kw)
        assert torch.equal(one[0], out[b]), b
        if lengths[b]:
            k, v = (x[table[b, :-(-lengths[b] // 16)].long()].flatten(0, 1)[:lengths[b]] for x in (kc, vc))
            want, _, tol, _ = ref.attention(q[b:b + 1], k, v, **kw)
            ref.assert_within(out[b:b + 1], want, tol, "sequence %d" % b)


def test_a_bad_length_far_back_and_a_replayed_graph():
    lengths = lengths_of(1300, "ragged")
    q, kc, vc, table, n = pages_of(lengths, 8, 2, 64, 16, 3)
    want = dg.det_attn_decode(q, kc, vc, table, n)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = dg.det_attn_decode(q, kc, vc, table, n)
    g.replay()
    assert torch.equal(got, want) and dg.det_gemm_check() == 0
    n[1290] = -1
    n[3] = 0
    g.replay()
    assert dg.det_gemm_check() == 1
    assert not got[1290].any() and not got[3].any()
    keep = [b for b in range(1300) if b not in (3, 1290)]
    assert torch.equal(got[keep], want[keep])
