"""The rows of the embedding's gradient that never occur, written by the sort's
launch (the first 128 MB) and by the gradient's: outputs hold NaN before, rows
that occur lie on both sides of the border, and what lies between the output's
rows is left alone."""
import pytest
import torch

import invariant_deterministic_gemm_gb300 as dg
import ops_ref as ref
from test_gpu_moe import rows_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,V,H,pad", [(1, 5, 8, 0), (0, 33, 64, 8), (333, 1003, 1000, 8), (70, 3, 7, 1), (40, 17, 2056, 8),
                                       (900, 40001, 1000, 8), (900, 70001, 1000, 0), (50, 131077, 1032, 8), (0, 70003, 1000, 8),
                                       (20, 9, 1 << 23, 0)])
def test_every_row_is_written(T, V, H, pad, dtype):
    es = torch.finfo(dtype).bits // 8
    border = (128 << 20) // (H * es)                           # rows zeroed beside the sort
    g = torch.Generator().manual_seed(T + V)
    tok = torch.randint(0, V, (T,), generator=g)
    if T > 8:
        tok[:8] = torch.tensor([0, V - 1, border - 1, border, border + 1, 1, V - 2, V // 2]).clamp(0, V - 1)
    dy = rows_of(T, H, 3, 0.1) if H < 1 << 20 else torch.ones(T, H, dtype=torch.bfloat16, device="cuda")
    ld = (H * es + 15) // 16 * 16 // es + pad // (es // 2) // (16 // es) * (16 // es)
    wide = torch.full((V, ld), float("nan"), dtype=dtype, device="cuda")
    out = wide[:, :H]
    got = dg.det_embedding_grad(dy, tok.cuda(), V, 1.7, out=out)
    assert dg.det_gemm_check() == 0
    assert got.data_ptr() == wide.data_ptr()
    assert torch.isnan(wide[:, H:]).all()
    seen = torch.zeros(V, dtype=torch.bool)
    seen[tok] = True
    assert not got[~seen.cuda()].any()
    s = float(torch.tensor(1.7, dtype=torch.float32))
    half = ref.EPS_F32 if dtype == torch.float32 else ref.EPS_BF16
    for v in torch.unique(tok).tolist():
        rows = dy[(tok == v).cuda()].double() * s
        want, size, n = rows.sum(0), rows.abs().sum(0), rows.shape[0]
        tol = size * (min(n, 32) + n // 32 + 2) * 2.0 ** -24
        assert ((got[v].double() - want).abs() <= tol + half * (want.abs() + tol)).all(), v
