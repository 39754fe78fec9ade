"""The attention operators as a model uses them together: a prompt through
the cache and packed attention, then token by token over the cache; and a
training step from projections to their gradients."""
import pytest
import torch

import attn_ref as ref
import invariant_deterministic_gemm_gb300 as dg
from test_gpu_rope import tables

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32


def randn(seed, *shape, std=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(BF16).cuda()


@pytest.mark.parametrize("kw", [dict(), dict(window=100, sinks=4)])
def test_prompt_and_next_tokens(kw):
    """Each token's output from the cache agrees with the whole sequence's at once; both are within BF16's bound
    of 64 bits on the same rotated keys."""
    H, KV, D, page, prompt, total = 8, 2, 128, 16, 300, 340
    x = randn(1, total, H + 2 * KV, D)
    q, k, v = x[:, :H], x[:, H:H + KV], x[:, H + KV:]
    c, s = tables(total, D)
    pos = torch.arange(total, dtype=I32).cuda()
    pages = -(-total // page)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(2)).to(I32).cuda()[None]
    slots = (table[0].long()[pos.long() // page] * page + pos.long() % page).to(I32)
    kc, vc = (torch.full((pages, page, KV, D), float("nan"), dtype=BF16, device="cuda") for _ in range(2))
    qp = dg.det_kv_append(q[:prompt], k[:prompt], v[:prompt], c, s, pos[:prompt].clone(), slots[:prompt].clone(), kc, vc)
    kr = dg.det_rope(k, c, s, pos)
    out, _ = dg.det_attn(qp, kr[:prompt], v[:prompt], **kw)
    rows = [out]
    for t in range(prompt, total):
        one = slice(t, t + 1)
        qt = dg.det_kv_append(q[one], k[one], v[one], c, s, pos[one].clone(), slots[one].clone(), kc, vc)
        rows.append(dg.det_attn_decode(qt, kc, vc, table, torch.tensor([t + 1], dtype=I32).cuda(), **kw))
    assert dg.det_gemm_check() == 0
    got, qr = torch.cat(rows), dg.det_rope(q, c, s, pos)
    want, _, tol, _ = ref.attention(qr, kr, v, **kw)
    ref.assert_within(got, want, tol)
    whole, _ = dg.det_attn(qr, kr, v, **kw)
    assert torch.equal(whole[:prompt], out)


def test_training_step_against_autograd():
    """From projections to their gradients: rotation, attention of packed documents, and back. Against autograd in
    64 bits of the same step without roundings: the rotated q and k, out, P and dS are rounded to BF16 on the way
    (2^-8 of each at most, 2^-9.5 in the mean square), so each gradient is off by a few of these in the 2-norm:
    2^-6 allows for eight in a row, all at their mean."""
    T, H, KV, D, rot = 260, 4, 2, 64, 32
    x, w = randn(1, T, H + 2 * KV, D), randn(2, T, H, D)
    c, s = tables(T, rot)
    lengths = (100, 37, 123)
    pos = torch.cat([torch.arange(n) for n in lengths]).to(I32).cuda()
    b = torch.tensor([0, 100, 137, 260], dtype=I32).cuda()
    q, k, v = x[:, :H], x[:, H:H + KV], x[:, H + KV:]
    kw = dict(window=40, sinks=3)
    qr, kr = dg.det_rope(q, c, s, pos), dg.det_rope(k, c, s, pos)
    out, lse = dg.det_attn(qr, kr, v, b, **kw)
    dq, dk, dv = dg.det_attn_bwd(w, qr, kr, v, out, lse, b, **kw)
    got = torch.cat([dg.det_rope(dq, c, s, pos, inverse=True), dg.det_rope(dk, c, s, pos, inverse=True), dv], 1)
    assert dg.det_gemm_check() == 0
    z = ref.f64(x).requires_grad_()
    co, si = ref.f64(c)[pos.cpu().long()][:, None], ref.f64(s)[pos.cpu().long()][:, None]
    lo, hi, rest = z[:, :H + KV, :rot // 2], z[:, :H + KV, rot // 2:rot], z[:, :H + KV, rot:]
    y = torch.cat([lo * co - hi * si, hi * co + lo * si, rest], -1)
    loss, a = 0.0, 0
    for n in lengths:
        vis = ref.visible(n, n, **kw)
        for h in range(H):
            g = h // (H // KV)
            sc = (y[a:a + n, h] @ y[a:a + n, H + g].T * D ** -0.5).masked_fill(~vis, -float("inf"))
            loss = loss + (torch.softmax(sc, 1) @ z[a:a + n, H + KV + g] * ref.f64(w)[a:a + n, h]).sum()
        a += n
    loss.backward()
    for part in (slice(0, H), slice(H, H + KV), slice(H + KV, None)):
        g, e = ref.f64(got)[:, part], z.grad[:, part]
        assert float((g - e).norm() / e.norm()) < 2.0 ** -6
