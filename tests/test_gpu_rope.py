"""Rotary positions and appending to a paged cache on the GPU against 64 bits."""
import pytest
import torch

import attn_ref as ref
import invariant_deterministic_gemm_gb300 as dg

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32


def tables(P, rot, base=10000.0):
    a = torch.arange(P, dtype=ref.F64)[:, None] * base ** (-torch.arange(0, rot, 2, dtype=ref.F64) / rot)
    return torch.cos(a).float().cuda(), torch.sin(a).float().cuda()


def randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(BF16).cuda()


def positions(T, P, seed=0):
    return torch.randint(0, P, (T,), generator=torch.Generator().manual_seed(seed), dtype=I32).cuda()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,D,rot", [(1, 1, 8, 8), (3, 5, 8, 2), (17, 32, 128, 128), (40, 3, 80, 40), (40, 3, 80, 80), (9, 4, 64, 16), (9, 4, 120, 6),
                                       (33, 2, 128, 126), (700, 7, 96, 24), (5, 200, 64, 64)])
def test_rotation_and_its_inverse(T, H, D, rot, interleaved):
    x = randn(T, T, H + 2, D)[:, 1:H + 1]
    c, s = tables(3000, rot)
    pos = positions(T, 3000)
    for inverse in (False, True):
        y = dg.det_rope(x, c, s, pos, interleaved=interleaved, inverse=inverse)
        ref.assert_within(y, *ref.turned(x, c, s, pos, interleaved, inverse))
        assert torch.equal(y[..., rot:], x[..., rot:])
    z = x.clone()
    assert dg.det_rope(z, c, s, pos, interleaved=interleaved, inverse=True, out=z).data_ptr() == z.data_ptr() and torch.equal(z, y)
    assert dg.det_gemm_check() == 0


def test_the_inverse_is_the_gradient():
    """<rope(x), w> = <x, inverse(w)>, and against differences: the rotation is linear."""
    T, H, D = 30, 4, 64
    x, w = randn(1, T, H, D), randn(2, T, H, D)
    c, s = tables(500, 48)
    pos = positions(T, 500)
    for inter in (False, True):
        y, ty = ref.turned(x, c, s, pos, inter)
        g = dg.det_rope(w, c, s, pos, interleaved=inter, inverse=True)
        lhs, rhs = float((y * ref.f64(w)).sum()), float((ref.f64(g) * ref.f64(x)).sum())
        assert abs(lhs - rhs) <= float((ref.turned(w, c, s, pos, inter, True)[1] * ref.f64(x).abs()).sum()) + 1e-9


def test_a_token_alone_has_the_same_bits():
    x = randn(3, 600, 12, 128)
    c, s = tables(600, 128)
    pos = positions(600, 600)
    y = dg.det_rope(x, c, s, pos)
    for t in (0, 77, 599):
        assert torch.equal(dg.det_rope(x[t:t + 1], c, s, pos[t:t + 1].clone()), y[t:t + 1])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,KV,D,rot,page", [(1, 1, 1, 64, 64, 1), (17, 32, 32, 128, 128, 16), (50, 8, 2, 80, 40, 7), (300, 3, 3, 96, 96, 64), (9, 16, 1, 24, 10, 8)])
def test_append(T, H, KV, D, rot, page, interleaved):
    x = randn(T, T, H + 2 * KV, D)
    q, k, v = x[:, :H], x[:, H:H + KV], x[:, H + KV:]
    c, s = tables(1000, rot)
    pos = positions(T, 1000)
    pages = -(-T // page) + 2
    g = torch.Generator().manual_seed(T)
    slots = torch.randperm(pages * page, generator=g)[:T].to(I32)
    slots[torch.rand(T, generator=g) < 0.2] = -1
    kc, vc = randn(1, pages, page, KV, D), randn(2, pages, KV, page, D).transpose(1, 2)      # two layouts
    wk, wv = kc.clone(), vc.clone()
    out = dg.det_kv_append(q, k, v, c, s, pos, slots.cuda(), kc, vc, interleaved=interleaved)
    assert dg.det_gemm_check() == 0
    assert torch.equal(out, dg.det_rope(q, c, s, pos, interleaved=interleaved))
    ref.assert_within(out, *ref.turned(q, c, s, pos, interleaved))
    kr = dg.det_rope(k, c, s, pos, interleaved=interleaved)
    for t, at in enumerate(slots.tolist()):
        if at >= 0:
            wk[at // page, at % page], wv[at // page, at % page] = kr[t], v[t]
    assert torch.equal(kc, wk) and torch.equal(vc, wv)
    kc2, vc2 = randn(1, pages, page, KV, D), randn(2, pages, KV, page, D).transpose(1, 2)
    assert dg.det_kv_append(None, k, v, c, s, pos, slots.cuda(), kc2, vc2, interleaved=interleaved) is None
    assert torch.equal(kc2, wk) and torch.equal(vc2, wv)


def test_positions_and_slots_outside_are_reported_and_store_nothing():
    T, KV, D = 6, 2, 64
    q, k, v = randn(1, T, 4, D), randn(2, T, KV, D), randn(3, T, KV, D)
    c, s = tables(100, 64)
    pos = torch.tensor([0, 99, 100, -1, 5, 7], dtype=I32).cuda()
    y = dg.det_rope(q, c, s, pos)
    assert dg.det_gemm_check() == 1
    assert not y[2:4].any() and y[1].any()
    kc, vc = randn(4, 3, 8, KV, D), randn(5, 3, 8, KV, D)
    wk, wv = kc.clone(), vc.clone()
    slots = torch.tensor([-1, -1, 3, 4, 24, -2], dtype=I32).cuda()
    dg.det_kv_append(q, k, v, c, s, pos, slots, kc, vc)
    assert dg.det_gemm_check() == 1
    assert torch.equal(kc, wk) and torch.equal(vc, wv)
    slots[:] = torch.tensor([0, 1, 2, 3, 23, -1], dtype=I32)
    dg.det_kv_append(q, k, v, c, s, pos.clamp(0, 99), slots, kc, vc)
    assert dg.det_gemm_check() == 0
    assert torch.equal(vc[2, 7], v[4])


def test_values_that_are_not_finite_pass_through():
    x = randn(1, 4, 2, 64)
    x[1, 0, 3], x[2, 1, 40] = float("inf"), float("nan")
    c, s = tables(10, 32)
    pos = torch.tensor([1, 2, 3, 4], dtype=I32).cuda()
    y = dg.det_rope(x, c, s, pos).float()
    assert torch.isfinite(y[0]).all() and torch.isfinite(y[3]).all() and not torch.isfinite(y[1, 0, [3, 19]]).any()
    assert torch.isnan(y[2, 1, 40]) and torch.isfinite(y[2, 0]).all()


def test_empty():
    c, s = tables(10, 32)
    none = torch.zeros(0, dtype=I32).cuda()
    assert dg.det_rope(randn(1, 0, 2, 64), c, s, none).shape == (0, 2, 64)
    kc, vc = randn(4, 3, 8, 2, 64), randn(5, 3, 8, 2, 64)
    dg.det_kv_append(randn(1, 0, 4, 64), randn(1, 0, 2, 64), randn(1, 0, 2, 64), c, s, none, none, kc, vc)
    assert dg.det_gemm_check() == 0
