"""The embedding lookup and its gradient on the GPU against 64-bit sums:
tokens that occur once, in chunks and in long runs, tokens outside the
table, padding, odd sizes, both gradient types, accumulation, and offsets
beyond 32 bits."""
import numpy as np
import pytest
import torch

import invariant_deterministic_gemm_gb300 as dg
import ops_ref as ref
from test_gpu_moe import rows_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,V,H,scale,dtype", [(1, 5, 8, 1.0, torch.int64), (17, 1000, 4096, 1.0, torch.int32),
                                               (333, 32003, 1000, 31.622776, torch.int64), (70, 3, 7, 0.3, torch.int32),
                                               (0, 4, 16, 1.0, torch.int64)])
def test_lookup(T, V, H, scale, dtype):
    table = rows_of(V, H, 1)
    tok = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(T)).to(dtype)
    out = dg.det_embedding(tok.cuda(), table, scale)
    assert dg.det_gemm_check() == 0
    want = ref.f64(table)[tok.numpy()] * np.float64(np.float32(scale))
    # one FP32 product and one rounding to BF16
    assert (np.abs(ref.f64(out) - want) <= np.abs(want) * (ref.EPS_BF16 + 2.0 ** -23)).all()


def test_lookup_of_a_token_outside_the_table_is_zero_and_reported():
    table = rows_of(10, 64, 2)
    out = dg.det_embedding(torch.tensor([3, 10, -1, 9]).cuda(), table)
    assert dg.det_gemm_check() == 1
    assert dg.det_gemm_check() == 0
    assert torch.equal(out[0], table[3]) and torch.equal(out[3], table[9])
    assert not out[1:3].any()


def tokens_of(kind, T, V):
    g = torch.Generator().manual_seed(T * 7 + V)
    if kind == "uniform":
        return torch.randint(0, V, (T,), generator=g)
    if kind == "one":
        return torch.full((T,), V - 1)
    if kind == "zipf":
        p = 1.0 / (torch.arange(V, dtype=torch.float64) + 2.7)
        return torch.multinomial(p, T, replacement=True, generator=g)
    return torch.arange(T) % V                                  # "cycle"


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind,T,V,H", [("uniform", 1, 5, 8), ("uniform", 333, 1003, 1000), ("one", 32, 9, 72), ("one", 33, 9, 72),
                                        ("one", 5000, 600, 40), ("zipf", 9000, 5000, 136), ("cycle", 640, 20, 7), ("cycle", 66, 2, 2056),
                                        ("zipf", 3001, 300000, 16), ("uniform", 0, 33, 64)])
def test_gradient(kind, T, V, H, out_dtype):
    tok = tokens_of(kind, T, V)
    dy = rows_of(T, H, 3, 0.1)
    scale = 1.7
    got = dg.det_embedding_grad(dy, tok.cuda(), V, scale, out_dtype=out_dtype)
    again = dg.det_embedding_grad(dy, tok.int().cuda(), V, scale, out_dtype=out_dtype)
    assert dg.det_gemm_check() == 0
    assert torch.equal(got, again)
    want, size = np.zeros((V, H)), np.zeros((V, H))
    s = float(np.float32(scale))
    np.add.at(want, tok.numpy(), ref.f64(dy) * s)
    np.add.at(size, tok.numpy(), np.abs(ref.f64(dy)) * s)
    n = np.bincount(tok.numpy(), minlength=V)[:, None]
    # 32 additions inside a chunk, one for each chunk, the scale; one rounding
    tol = size * (np.minimum(n, 32) + n // 32 + 2) * 2.0 ** -24
    half = ref.EPS_F32 if out_dtype == torch.float32 else ref.EPS_BF16
    assert (np.abs(ref.f64(got) - want) <= tol + half * (np.abs(want) + tol)).all()
    if T:                                                       # differences: the lookup is linear in the table
        v, c = int(tok[0]), H - 1
        slope = float((ref.f64(dy)[:, c] * (tok.numpy() == v) * s).sum())
        assert abs(ref.f64(got)[v, c] - slope) <= tol[v, c] + half * (abs(slope) + tol[v, c])


def test_gradient_of_a_row_depends_on_its_own_occurrences_alone():
    V, H = 50, 264
    g = torch.Generator().manual_seed(5)
    tok = torch.randint(0, 4, (900,), generator=g)
    dy = rows_of(900, H, 9)
    full = dg.det_embedding_grad(dy, tok.cuda(), V)
    alone = dg.det_embedding_grad(dy[tok.cuda() == 2].contiguous(), tok[tok == 2].cuda(), V)
    moved = dg.det_embedding_grad(dy, torch.where(tok == 2, tok, tok + 40).cuda(), V)
    assert torch.equal(full[2].view(torch.int32), alone[2].view(torch.int32))
    assert torch.equal(full[2].view(torch.int32), moved[2].view(torch.int32))


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_accumulate_padding_and_bad_tokens(out_dtype):
    V, H, T = 40, 100, 500
    tok = tokens_of("zipf", T, V)
    dy = rows_of(T, H, 4, 0.1)
    base = torch.randn(V, H, generator=torch.Generator().manual_seed(1)).to(out_dtype)
    per = 16 // base.element_size()
    buf = torch.zeros(V, (H + per - 1) // per * per, dtype=out_dtype).cuda()[:, :H]
    buf.copy_(base)
    dg.det_embedding_grad(dy, tok.cuda(), V, 2.0, padding_idx=1, out=buf, accumulate=True)
    assert dg.det_gemm_check() == 0
    keep = tok != 1
    want, size = ref.f64(base), np.abs(ref.f64(base))
    np.add.at(want, tok[keep].numpy(), ref.f64(dy)[keep.numpy()] * 2.0)
    np.add.at(size, tok[keep].numpy(), np.abs(ref.f64(dy)[keep.numpy()]) * 2.0)
    n = np.bincount(tok.numpy(), minlength=V)[:, None]
    tol = size * (np.minimum(n, 32) + n // 32 + 3) * 2.0 ** -24
    half = ref.EPS_F32 if out_dtype == torch.float32 else ref.EPS_BF16
    assert (np.abs(ref.f64(buf) - want) <= tol + half * (np.abs(want) + tol)).all()
    assert torch.equal(buf[1].cpu(), base[1])
    bad = tok.clone()
    bad[3], bad[4] = V, -7
    got = dg.det_embedding_grad(dy, bad.cuda(), V)
    assert dg.det_gemm_check() == 1
    good = torch.ones(T, dtype=torch.bool)
    good[3:5] = False
    rest = torch.zeros(T - 2, 104, dtype=torch.bfloat16, device="cuda")[:, :H]      # 16-byte row pitch
    rest.copy_(dy[good.cuda()])
    want = dg.det_embedding_grad(rest, tok[good].cuda(), V)
    assert torch.equal(got, want) and dg.det_gemm_check() == 0


@pytest.mark.slow
def test_rows_beyond_32_bit_offsets():
    V, H = 151936, 32768                                        # 5.0e9 elements
    table = torch.empty((V, H), dtype=torch.bfloat16, device="cuda")
    table[-3:] = rows_of(3, H, 1)
    table[0] = 1.0
    out = dg.det_embedding(torch.tensor([V - 1, 0, V - 3]).cuda(), table)
    assert torch.equal(out[0], table[-1]) and torch.equal(out[2], table[-3])
    dy = rows_of(40, H, 2)
    tok = torch.full((40,), V - 1)
    tok[7] = 0
    got = dg.det_embedding_grad(dy, tok.cuda(), V, out=table)
    assert dg.det_gemm_check() == 0
    assert torch.equal(got[0], dy[7])
    small = dg.det_embedding_grad(dy[tok.cuda() != 0].contiguous(), torch.ones(39, dtype=torch.int64).cuda(), 2,
                                  out_dtype=torch.bfloat16)
    assert torch.equal(got[-1], small[1]) and not got[V // 2].any() and not got[-2].any()
