"""Bounds that go down or leave the rows: each of the packed operators reports them."""
import pytest
import torch

import invariant_deterministic_gemm_gb300 as dg
from test_gpu_attn import make

pytestmark = pytest.mark.gpu


def on_gpu(b):
    return torch.tensor(b, dtype=torch.int32).cuda()


BAD = [([0, 60], None), ([-3, 50], None), ([0, 30, 20, 50], None), ([10, 5], None), ([0, 30, 50], [0, 20, 10]), ([0, 50], [0, 51]),
       ([0, 20, 50], [-1, 20, 50]), ([0] * 100 + [1 << 30] + [50], None)]


@pytest.mark.parametrize("b,kb", BAD)
def test_both_passes_report_bad_bounds(b, kb):
    q, k, v = make(50, 50, 2, 1, 64, 16)
    b, kb = on_gpu(b), None if kb is None else on_gpu(kb)
    out, lse = dg.det_attn(q, k, v)
    assert dg.det_gemm_check() == 0
    dg.det_attn(q, k, v, b, kb)
    assert dg.det_gemm_check() == 1
    dg.det_attn_bwd(out, q, k, v, out, lse, b, kb)
    assert dg.det_gemm_check() == 1
    good = on_gpu([0, 50])
    dg.det_attn_bwd(out, q, k, v, out, lse, good)
    assert dg.det_gemm_check() == 0


@pytest.mark.parametrize("kb,status", [([0, 5, 50], 0), ([0, 5, 51], 1), ([0, 60, 50], 1)])
def test_gradients_without_queries_report_the_keys_bounds(kb, status):
    q, k, v = make(50, 50, 2, 1, 64, 16)
    q, lse = q[:0], torch.empty((2, 0), device="cuda")
    _, dk, dv = dg.det_attn_bwd(q, q, k, v, q, lse, on_gpu([0, 0, 0]), on_gpu(kb))
    assert dg.det_gemm_check() == status
    assert not dk.any() and not dv.any()
