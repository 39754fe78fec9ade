"""The e4m3 quantisers and block-scaled products on the GPU against 64-bit
implementations: quantised values and scales exactly, products bit for bit
on exact inputs and within derived bounds on real ones, every tile, ragged
sizes, groups of any size (empty ones too), both output types, gradients,
bits that do not depend on the batch, and a timeout."""
import numpy as np
import pytest
import torch

import invariant_deterministic_gemm_gb300 as dg
import ops_ref as ref
from test_gpu_moe import rows_of

pytestmark = pytest.mark.gpu


def ok():
    assert dg.det_gemm_check() == 0


def real(M, K, seed):
    x = rows_of(M, K, seed)
    x[:, :: max(1, K // 7)] *= 20
    return x


@pytest.mark.parametrize("M,K", [(1, 128), (3, 4096), (17, 1000), (5, 7), (130, 264), (2, 2056)])
def test_quantize_rows(M, K):
    x = real(M, K, M + K)
    if M > 2:
        x[1] = 0
        x[2] *= 2.0 ** -40
    q, s = dg.det_fp8_quantize_rows(x)
    ok()
    rq, rs = ref.quantize(ref.f64(x))
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(ref.f64(q.float()), rq)
    # gathered: the same rows, zeros where there is none
    rows = torch.tensor([2 * M - 1, 0, -1, 2 * M + 4], dtype=torch.int32)
    q2, s2 = dg.det_fp8_quantize_rows(x, rows.cuda(), 2)
    ok()
    assert torch.equal(q2[0].float(), q[M - 1].float()) and torch.equal(q2[1].float(), q[0].float())
    assert torch.equal(s2[0], s[M - 1]) and not q2[2:].float().any()


def test_every_ratio_of_two_bf16_values_rounds_as_in_64_bits():
    """All 128 x 128 ratios of BF16 significands, ties among them."""
    m = torch.arange(128, 256).float()
    x = torch.zeros(128 * 4, 256)
    for i in range(4):
        x[128 * i:128 * (i + 1), :128] = m[None, :] * 2.0 ** -(i * 5) / 256
    x[:, 0] = (m[torch.arange(512) % 128]) / 64                 # the block's maximum
    x[:, 128:] = -x[:, :128]
    x = x.bfloat16().cuda()
    q, s = dg.det_fp8_quantize_rows(x)
    rq, rs = ref.quantize(ref.f64(x))
    assert np.array_equal(ref.f64(q.float()), rq) and np.array_equal(s.cpu().numpy(), rs)
    qt, st = dg.det_fp8_quantize_cols(x.t().contiguous())
    assert np.array_equal(ref.f64(qt.float()), rq) and np.array_equal(st.t().cpu().numpy(), rs)
    ok()


def test_extreme_blocks():
    x = torch.zeros(6, 256)
    x[0, :4] = torch.tensor([3e38, -1e38, 1e30, 1.0])           # 448 x would overflow
    x[1, 0] = 2.0 ** -120                                       # below the smallest scale
    x[2, 5] = float("inf")
    x[3, 200] = float("nan")
    x[4, :3] = torch.tensor([2.0 ** -99, 2.0 ** -108, -(2.0 ** -102)])
    x = x.bfloat16()
    q, s = dg.det_fp8_quantize_rows(x.cuda())
    ok()
    assert torch.isnan(s[2, 0]) and torch.isnan(s[3, 1]) and not q[2].float().any() and not q[3].float().any()
    fine = [0, 1, 4, 5]
    rq, rs = ref.quantize(ref.f64(x[fine]))
    assert np.array_equal(ref.f64(q[fine].float()), rq) and np.array_equal(s[fine].cpu().numpy(), rs)
    w = torch.eye(128, 256).bfloat16().cuda()
    wq, ws = dg.det_fp8_quantize_tiles(w)
    y = dg.det_fp8_gemm(q, s, wq, ws)
    ok()
    assert torch.isnan(y[2:4]).all() and torch.isfinite(y[fine]).all()


@pytest.mark.parametrize("M,K,bounds", [(1, 64, None), (300, 100, None), (128, 7, None), (257, 1000, None),
                                        (300, 136, [0, 10, 10, 139, 300]), (500, 72, [3, 131, 400, 400, 470]), (5, 64, [0, 0, 5])])
def test_quantize_cols(M, K, bounds):
    x = real(M, K, M)
    off = None if bounds is None else torch.tensor(bounds, dtype=torch.int32).cuda()
    q, s = dg.det_fp8_quantize_cols(x, off)
    ok()
    X, at = ref.f64(x), 0
    for lo, hi in ([(0, M)] if bounds is None else zip(bounds[:-1], bounds[1:])):
        nb = (hi - lo + 127) // 128
        if nb == 0:
            continue
        rq, rs = ref.quantize(X[lo:hi], axis=0)
        got = ref.f64(q[:, at * 128:(at + nb) * 128].float()).T
        assert np.array_equal(got[:hi - lo], rq) and not got[hi - lo:].any()
        assert np.array_equal(s[at:at + nb].cpu().numpy(), rs)
        at += nb


@pytest.mark.parametrize("shape", [(128, 128), (130, 264), (7, 1000), (3, 200, 136), (2, 16, 16), (1, 129, 7)])
def test_quantize_tiles(shape):
    g = torch.Generator().manual_seed(sum(shape))
    K = shape[-1]
    wide = torch.zeros(shape[:-1] + ((K + 7) // 8 * 8 + 8,), dtype=torch.bfloat16)
    wide[..., :K] = torch.randn(shape, generator=g) * 0.02
    w = wide.cuda()[..., :K]
    q, s = dg.det_fp8_quantize_tiles(w)
    qt, st = dg.det_fp8_quantize_tiles(w, transposed=True)
    ok()
    for i in range(shape[0] if len(shape) == 3 else 1):
        pick = (lambda t: t[i]) if len(shape) == 3 else (lambda t: t)
        rq, rs = ref.quantize_tiles(ref.f64(pick(w)))
        assert np.array_equal(ref.f64(pick(q).float()), rq) and np.array_equal(pick(s).cpu().numpy(), rs)
        assert np.array_equal(ref.f64(pick(qt).float()), rq.T) and np.array_equal(pick(st).cpu().numpy(), rs.T)


def exact_operand(M, K, seed):
    """Integers of at most 4 in e4m3 and scales that are powers of two: every sum is exact in FP32."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(-4, 5, (M, K), generator=g).double().numpy()
    nb = (K + 127) // 128
    s = torch.pow(2.0, torch.randint(-2, 3, (M, nb), generator=g).float())
    return q, s


SHAPES = [(1, 128, 128), (1, 32, 16), (3, 1000, 4096), (16, 130, 264), (17, 40, 7), (33, 257, 1000), (64, 200, 2056), (65, 300, 640),
          (128, 128, 128), (130, 136, 520), (200, 1000, 1032), (300, 64, 4096), (1021, 520, 300), (129, 4000, 136), (2500, 2600, 260)]


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_is_exact_on_exact_inputs(M, N, K, out_dtype):
    qa, sa = exact_operand(M, K, M)
    qw, _ = exact_operand(N, K, N + 1)
    g = torch.Generator().manual_seed(3)
    sw = torch.pow(2.0, torch.randint(-2, 3, ((N + 127) // 128, (K + 127) // 128), generator=g).float())
    A, W = ref.e4m3_tensor(qa).cuda()[:, :K], ref.e4m3_tensor(qw).cuda()[:, :K]
    C = dg.det_fp8_gemm(A, sa.cuda(), W, sw.cuda(), out_dtype=out_dtype)
    ok()
    want = torch.from_numpy(ref.dequantize(qa, sa.numpy())) @ torch.from_numpy(ref.dequantize_tiles(qw, sw.numpy())).T
    assert torch.equal(C.cpu(), want.to(out_dtype))


@pytest.mark.parametrize("M,N,K", [(3, 300, 4096), (40, 500, 1000), (64, 512, 2000), (300, 700, 4096), (129, 130, 264)])
def test_product_of_quantised_tensors(M, N, K):
    x = real(M, K, 1)
    w = rows_of(N, K, 2, 0.02)
    q, s = dg.det_fp8_quantize_rows(x)
    wq, ws = dg.det_fp8_quantize_tiles(w)
    for out_dtype in (torch.float32, torch.bfloat16):
        C = dg.det_fp8_gemm(q, s, wq, ws, out_dtype=out_dtype)
        ok()
        a = ref.dequantize(*ref.quantize(ref.f64(x)))
        b = ref.dequantize_tiles(*ref.quantize_tiles(ref.f64(w)))
        want = a @ b.T
        tol = ref.product_tolerance(np.abs(a) @ np.abs(b).T, (K + 127) // 128, out_dtype, want)
        assert (np.abs(ref.f64(C) - want) <= tol).all()


@pytest.mark.parametrize("K", [100, 640, 1416, 2688])
@pytest.mark.parametrize("M,N", [(5, 3000), (5, 12000), (5, 20000), (20, 3000), (20, 12000), (20, 20000), (50, 3000), (50, 8000), (50, 12000)])
def test_few_rows_on_every_weight_tile(M, N, K):
    """Weight tiles of 32, 64 and 128 rows beside 16, 32 and 64 tokens, with
    odd and even numbers of blocks, more than one tile for some CTAs."""
    qa, sa = exact_operand(M, K, M)
    qw, _ = exact_operand(N, K, N + 1)
    g = torch.Generator().manual_seed(3)
    sw = torch.pow(2.0, torch.randint(-2, 3, ((N + 127) // 128, (K + 127) // 128), generator=g).float())
    A, W = ref.e4m3_tensor(qa).cuda()[:, :K], ref.e4m3_tensor(qw).cuda()[:, :K]
    want = torch.from_numpy(ref.dequantize(qa, sa.numpy())) @ torch.from_numpy(ref.dequantize_tiles(qw, sw.numpy())).T
    for _ in range(3):
        C = dg.det_fp8_gemm(A, sa.cuda(), W, sw.cuda(), out_dtype=torch.float32)
        ok()
        assert torch.equal(C.cpu(), want.float())


@pytest.mark.parametrize("T,E,N,K", [(4, 16, 2048, 1400), (132, 16, 2048, 4096), (132, 16, 1000, 640), (250, 16, 2048, 1400), (900, 16, 1500, 900),
                                     (60, 64, 700, 1400)])
def test_few_rows_for_each_of_many_experts(T, E, N, K):
    x = real(T, K, 1)
    w = torch.zeros(E, N, (K + 7) // 8 * 8, dtype=torch.bfloat16, device="cuda")[:, :, :K]
    for e in range(E):
        w[e] = rows_of(N, K, 10 + e, 0.02)
    q, s = dg.det_fp8_quantize_rows(x)
    wq, ws = dg.det_fp8_quantize_tiles(w)
    g = torch.Generator().manual_seed(T)
    cuts = torch.sort(torch.randint(0, T + 1, (E - 1,), generator=g))[0]
    bounds = [0] + cuts.tolist() + [T]
    off = torch.tensor(bounds, dtype=torch.int32).cuda()
    a, b = ref.dequantize(*ref.quantize(ref.f64(x))), None
    for _ in range(3):
        C = dg.det_fp8_gemm_grouped(q, s, wq, ws, off, out_dtype=torch.float32)
        ok()
        for e, (lo, hi) in enumerate(zip(bounds[:-1], bounds[1:])):
            if hi > lo:
                b = ref.dequantize_tiles(*ref.quantize_tiles(ref.f64(w[e])))
                want = a[lo:hi] @ b.T
                tol = ref.product_tolerance(np.abs(a[lo:hi]) @ np.abs(b).T, (K + 127) // 128, torch.float32, want)
                assert (np.abs(ref.f64(C[lo:hi]) - want) <= tol).all(), e


def test_bounds_made_by_the_launch_in_front_are_read_after_it():
    """Group bounds from the kernel directly before the product."""
    x = real(300, 256, 1)
    w = torch.stack([rows_of(200, 256, 10 + g, 0.02).contiguous() for g in range(4)])
    q, s = dg.det_fp8_quantize_rows(x)
    wq, ws = dg.det_fp8_quantize_tiles(w)
    counts = torch.tensor([0, 7, 130, 0, 163], device="cuda")
    want = dg.det_fp8_gemm_grouped(q, s, wq, ws, torch.tensor([0, 7, 137, 137, 300], dtype=torch.int32).cuda())
    for _ in range(20):
        off = torch.cumsum(counts, 0, dtype=torch.int32)
        assert torch.equal(dg.det_fp8_gemm_grouped(q, s, wq, ws, off), want)
    ok()


def test_an_empty_contraction_is_zero():
    q = torch.zeros(5, 16, device="cuda").to(torch.float8_e4m3fn)[:, :0]
    w = torch.zeros(24, 16, device="cuda").to(torch.float8_e4m3fn)[:, :0]
    C = dg.det_fp8_gemm(q, torch.zeros(5, 0).cuda(), w, torch.zeros(1, 0).cuda())
    ok()
    assert C.shape == (5, 24) and not C.any()


def test_rows_have_the_same_bits_in_every_batch_and_every_tile():
    M, N, K = 700, 1100, 2300
    x = real(M, K, 8)
    q, s = dg.det_fp8_quantize_rows(x)
    wq, ws = dg.det_fp8_quantize_tiles(rows_of(N, K, 9, 0.02))
    full = dg.det_fp8_gemm(q, s, wq, ws, out_dtype=torch.float32)
    for m in (1, 2, 16, 17, 32, 33, 64, 65, 128, 300):
        for lo in (0, 5):
            part = dg.det_fp8_gemm(q[lo:lo + m], s[lo:lo + m], wq, ws, out_dtype=torch.float32)
            assert torch.equal(part.view(torch.int32), full[lo:lo + m].view(torch.int32)), (m, lo)
    for n in (32, 100, 128, 200):
        part = dg.det_fp8_gemm(q, s, wq[:n], ws[:(n + 127) // 128], out_dtype=torch.float32)
        assert torch.equal(part.view(torch.int32), full[:, :n].contiguous().view(torch.int32)), n
    ok()


GROUPS = [(34, 256, 512, [0, 3, 3, 20, 34]), (1, 64, 64, [0, 0, 1]), (300, 200, 264, [0, 1, 130, 130, 290]), (700, 1000, 300, [5, 300, 301, 650]),
          (900, 300, 520, [0, 0, 900, 900]), (64, 136, 1000, [0] + [2 * i for i in range(1, 33)]), (40, 72, 128, [0, 0, 0, 0]),
          (2000, 520, 260, [0, 700, 1400, 1999])]


@pytest.mark.parametrize("M,N,K,bounds", GROUPS)
def test_grouped_product_is_each_groups_own_product(M, N, K, bounds):
    G = len(bounds) - 1
    x = real(M, K, 1)
    w = torch.stack([rows_of(N, K, 10 + g, 0.02).contiguous() for g in range(G)]) if K % 8 == 0 else None
    if w is None:
        w = torch.zeros(G, N, (K + 7) // 8 * 8, dtype=torch.bfloat16, device="cuda")[:, :, :K]
        for g in range(G):
            w[g] = rows_of(N, K, 10 + g, 0.02)
    q, s = dg.det_fp8_quantize_rows(x)
    wq, ws = dg.det_fp8_quantize_tiles(w)
    off = torch.tensor(bounds, dtype=torch.int32).cuda()
    for out_dtype in (torch.float32, torch.bfloat16):
        C = dg.det_fp8_gemm_grouped(q, s, wq, ws, off, out_dtype=out_dtype)
        ok()
        for g, (lo, hi) in enumerate(zip(bounds[:-1], bounds[1:])):
            if hi > lo:
                want = dg.det_fp8_gemm(q[lo:hi], s[lo:hi], wq[g], ws[g], out_dtype=out_dtype)
                assert torch.equal(C[lo:hi], want), g
        assert not C[:bounds[0]].any() and not C[bounds[-1]:].any()


def test_group_bounds_that_make_no_sense_are_reported_and_harmless():
    q, s = dg.det_fp8_quantize_rows(real(100, 256, 1))
    wq, ws = dg.det_fp8_quantize_tiles(torch.zeros(3, 64, 256, dtype=torch.bfloat16).cuda())
    for bounds in ([0, 50, 20, 100], [0, 50, 90, 1000], [-4, 50, 60, 100]):
        off = torch.tensor(bounds, dtype=torch.int32).cuda()
        dg.det_fp8_gemm_grouped(q, s, wq, ws, off)
        assert dg.det_gemm_check() == 1
    ok()


@pytest.mark.parametrize("M,N,K,bounds", [(1, 16, 16, None), (300, 264, 136, None), (128, 40, 1000, None), (1000, 130, 70, None), (700, 600, 520, None),
                                          (300, 136, 264, [0, 10, 10, 139, 300]), (500, 40, 72, [3, 131, 400, 400, 470]),
                                          (900, 300, 200, [0, 0, 900]), (2000, 260, 1032, [0, 700, 1400, 1999])])
def test_weight_gradient(M, N, K, bounds):
    dy, x = rows_of(M, N, 1, 1e-3), real(M, K, 2)
    off = None if bounds is None else torch.tensor(bounds, dtype=torch.int32).cuda()
    yt, sy = dg.det_fp8_quantize_cols(dy, off)
    xt, sx = dg.det_fp8_quantize_cols(x, off)
    for out_dtype in (torch.float32, torch.bfloat16):
        dW = dg.det_fp8_gemm_wgrad(yt, sy, xt, sx, off, out_dtype=out_dtype)
        ok()
        for g, (lo, hi) in enumerate([(0, M)] if bounds is None else list(zip(bounds[:-1], bounds[1:]))):
            got = ref.f64(dW if bounds is None else dW[g])
            if hi == lo:
                assert not got.any()
                continue
            a = ref.dequantize(*(v.T for v in ref.quantize(ref.f64(dy)[lo:hi], axis=0)))
            b = ref.dequantize(*(v.T for v in ref.quantize(ref.f64(x)[lo:hi], axis=0)))
            want = a @ b.T
            tol = ref.product_tolerance(np.abs(a) @ np.abs(b).T, (hi - lo + 127) // 128, out_dtype, want)
            assert (np.abs(got - want) <= tol).all(), g


def test_gradients_against_differences():
    """C = X W^T with the quantised operands' values: the products that give dX
    and dW, fed exact operands, are the slopes of <dC, C>."""
    M, N, K = 96, 160, 256
    qx, sx = exact_operand(M, K, 1)
    qw, _ = exact_operand(N, K, 2)
    qg, sg = exact_operand(M, N, 3)
    sw = torch.pow(2.0, torch.arange(4).float().reshape(2, 2) - 2)
    X, G = ref.dequantize(qx, sx.numpy()), ref.dequantize(qg, sg.numpy())
    Wd = ref.dequantize_tiles(qw, sw.numpy())
    dX = dg.det_fp8_gemm(ref.e4m3_tensor(qg).cuda(), sg.cuda(), ref.e4m3_tensor(qw.T).cuda(), sw.t().contiguous().cuda(),
                         out_dtype=torch.float32)
    f = lambda x, w: float((G * (x @ w.T)).sum())
    for m, k in ((0, 0), (95, 255), (40, 130)):
        xp, xm = X.copy(), X.copy()
        xp[m, k] += 1.0
        xm[m, k] -= 1.0
        assert float(dX[m, k]) == (f(xp, Wd) - f(xm, Wd)) / 2
    # integers of at most 4 over 128 tokens quantise to themselves where 4 is present: s = 4 / 448, q = 112 x
    x = torch.from_numpy(qx).bfloat16().cuda()
    g = torch.from_numpy(qg).bfloat16().cuda()
    yt, sy = dg.det_fp8_quantize_cols(g)
    xt, sxx = dg.det_fp8_quantize_cols(x)
    dW = dg.det_fp8_gemm_wgrad(yt, sy, xt, sxx)
    ok()
    a = ref.dequantize(*(v.T for v in ref.quantize(qg, axis=0)))
    b = ref.dequantize(*(v.T for v in ref.quantize(qx, axis=0)))
    h = lambda w: float((a.T * (b.T @ w.T)).sum())
    for n, k in ((0, 0), (159, 255), (77, 200)):
        wp, wm = Wd.copy(), Wd.copy()
        wp[n, k] += 1.0
        wm[n, k] -= 1.0
        slope = (h(wp) - h(wm)) / 2
        tol = np.abs(a[n]) @ np.abs(b[k]) * (128 * 2.0 ** -23 + 2.0 ** -20) + 1e-10 * abs(h(Wd))
        assert abs(float(dW[n, k]) - slope) <= tol


def test_timeout_is_reported_and_the_context_stays_usable():
    q, s = dg.det_fp8_quantize_rows(real(300, 1024, 1))
    wq, ws = dg.det_fp8_quantize_tiles(rows_of(600, 1024, 2, 0.02))
    want = dg.det_fp8_gemm(q, s, wq, ws)
    few = dg.det_fp8_gemm(q[:9], s[:9], wq, ws)
    ok()
    dg.det_ops_debug_force_timeout(True)
    try:
        dg.det_fp8_gemm(q, s, wq, ws)
        assert dg.det_gemm_check() == 6
        dg.det_fp8_gemm(q[:9], s[:9], wq, ws)
        assert dg.det_gemm_check() == 6
    finally:
        dg.det_ops_debug_force_timeout(False)
    assert torch.equal(dg.det_fp8_gemm(q, s, wq, ws), want)
    assert torch.equal(dg.det_fp8_gemm(q[:9], s[:9], wq, ws), few)
    ok()


def test_products_on_another_stream_and_in_a_graph():
    x = real(40, 512, 1)
    wq, ws = dg.det_fp8_quantize_tiles(rows_of(300, 512, 2, 0.02))

    def run(stream=None):
        q, s = dg.det_fp8_quantize_rows(x, stream=stream)
        return dg.det_fp8_gemm(q, s, wq, ws, stream=stream)

    want = run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = run(side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = run()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    ok()
