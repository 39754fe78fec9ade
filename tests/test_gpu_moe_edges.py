"""Routing on the GPU where FP32's range ends: biases of +inf and of the
lowest finite value, infinite logits, and groups whose values cancel."""
import numpy as np
import pytest
import torch

import invariant_deterministic_gemm_gb300 as dg
import ops_ref as ref
from test_gpu_moe import logits_of, ok, weight_tolerance

pytestmark = pytest.mark.gpu
INF = float("inf")


def check_route(x, k, bias, **kw):
    w, ids = dg.det_moe_route(x.cuda(), k, bias=None if bias is None else bias.cuda(), **kw)
    ok()
    rw, rids = ref.route(ref.f64(x), k, bias=None if bias is None else ref.f64(bias), **kw)
    assert np.array_equal(ids.cpu().numpy(), rids), (k, kw)
    assert (np.abs(ref.f64(w) - rw) <= weight_tolerance(rw, ref.f64(x))).all(), (k, kw)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,forced", [(8, [5]), (60, [0, 59]), (64, [33, 7, 12]), (256, [255]), (512, [3, 400])])
def test_experts_forced_by_an_infinite_bias(E, forced, score, dtype):
    """They come first, in the order of their indexes, with their own scores."""
    x = logits_of(33, E, dtype, E)
    x[1, forced[0]] = -INF                                     # masked all the same
    x[2] = -INF
    bias = (torch.rand(E, generator=torch.Generator().manual_seed(E)) - 0.5) * 0.2
    bias[forced] = INF
    for k in (1, 2, 4, 8):
        for renormalize in (True, False):
            check_route(x, k, bias, score=score, renormalize=renormalize)


def test_every_bias_infinite():
    x = logits_of(9, 40, torch.float32, 3)
    bias = torch.full((40,), INF)
    for k in (1, 6, 32):
        check_route(x, k, bias)
        check_route(x, k, bias, score="sigmoid")
