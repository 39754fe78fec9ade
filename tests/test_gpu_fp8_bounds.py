"""Group bounds that make no sense, on the GPU: every operator that reads them
reports them, and none computes with memory that nobody wrote."""
import pytest
import torch

import invariant_deterministic_gemm_gb300 as dg
from test_gpu_moe import rows_of

pytestmark = pytest.mark.gpu


def bounds_of(b):
    return torch.tensor(b, dtype=torch.int32).cuda()


def poison():
    """What the next allocations get holds e4m3 and FP32 NaNs."""
    torch.cuda.empty_cache()
    keep = [torch.full((1 << 19,), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(64)]
    keep += [torch.full((1 << 23,), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    del keep


def weight_gradient(dy, x, bounds):
    poison()
    off = bounds_of(bounds)
    yt, sy = dg.det_fp8_quantize_cols(dy, off)
    xt, sx = dg.det_fp8_quantize_cols(x, off)
    seen = dg.det_gemm_check()
    dW = dg.det_fp8_gemm_wgrad(yt, sy, xt, sx, off)
    dg.det_gemm_check()
    return seen, dW


@pytest.mark.parametrize("M,bad,same", [(100, [0, 100, 128], [0, 100, 100]), (200, [0, 130, 250], [0, 130, 200]), (100, [0, 101, 110, 120], [0, 100, 100, 100]),
                                        (129, [-5, 129, 1000], [0, 129, 129]), (300, [0] * 40 + [300, 1 << 30], [0] * 40 + [300, 300])])
def test_bounds_that_leave_the_matrix(M, bad, same):
    dy, x = rows_of(M, 136, 1, 1e-2), rows_of(M, 200, 2)
    seen, got = weight_gradient(dy, x, bad)
    assert seen == 1
    seen, want = weight_gradient(dy, x, same)
    assert seen == 0
    assert torch.equal(got, want)


@pytest.mark.parametrize("M,bounds", [(100, [0, 50, 20, 100]), (100, [30, 10, 100]), (300, [0, 300, 0, 300, 0, 300]), (260, [0, 400, 130, -7, 260]),
                                      (700, [0, 130, 129, 400, 131, 650]), (2000, [0] + [2000, 5] * 33), (9, [0, 4, 3, 9])])
def test_bounds_that_go_down_leave_zeros(M, bounds):
    """No row of a product has two owners: nothing is computed, and everything
    written. A weight gradient is made of what the quantiser wrote."""
    N, K, G = 200, 264, len(bounds) - 1
    x, dy = rows_of(M, K, 1), rows_of(M, N, 2, 1e-2)
    q, s = dg.det_fp8_quantize_rows(x)
    wq, ws = dg.det_fp8_quantize_tiles(torch.stack([rows_of(N, K, 10 + g, 0.02).contiguous() for g in range(G)]))
    out = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    dg.det_fp8_gemm_grouped(q, s, wq, ws, bounds_of(bounds), out=out)
    assert dg.det_gemm_check() == 1
    assert not out.any()
    seen, dW = weight_gradient(dy, x, bounds)
    assert seen == 1
    seen, again = weight_gradient(dy, x, bounds)
    assert torch.isfinite(dW).all() and torch.equal(dW, again)
