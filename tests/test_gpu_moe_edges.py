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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("offset", [0.0, 0.25])
def test_a_larger_logit_behind_exact_ties(offset, score, dtype):
    """Ten equal logits and a later one above them by one to three units in the
    last place: FP32 may give all of them one choice."""
    T, E = 200, 64
    g = torch.Generator().manual_seed(5)
    base = (torch.randn((T, 1), generator=g) * 2).to(dtype).float()
    x = base - 8.0 - torch.rand((T, E), generator=g)
    x[:, :10] = base
    step = torch.finfo(dtype).eps * 2.0 ** torch.floor(torch.log2(base.abs()))
    x[:, 40:41] = base + torch.randint(1, 4, (T, 1), generator=g) * step
    x = x.to(dtype)
    bias = torch.full((E,), offset)
    for k in (1, 2, 5, 10, 11):
        check_route(x, k, bias, score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_a_choice_with_a_large_bias_among_small_scores(score):
    """Scores of 1e-7 to 1e-6 that FP32 tells apart, and one of about a half
    whose bias leaves it among them, off by several of their distances in FP32."""
    T, E = 60, 64
    g = torch.Generator().manual_seed(9)
    for t in range(T):
        s = 1e-7 + 9e-7 * torch.rand(E, generator=g, dtype=torch.float64)
        s[10] = 0.3 + 0.4 * float(torch.rand(1, generator=g))
        if score == "softmax":
            s[11] = 1.0 - float(s[10]) - float(s[12:].sum()) - float(s[:10].sum())
            x = torch.log(s)
        else:
            x = torch.log(s / (1.0 - s))
        x = x.float()[None]
        true = torch.softmax(x.double(), 1)[0] if score == "softmax" else torch.sigmoid(x.double())[0]
        bias = torch.zeros(E)
        bias[10] = (5e-7 - true[10]).float()
        bias[11] = -INF
        for k in (4, 16, 28):
            check_route(x, k, bias, score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_close_choices_below_an_infinite_bias(score):
    x = logits_of(40, 64, torch.float32, 7)
    s = torch.softmax(x.double(), 1) if score == "softmax" else torch.sigmoid(x.double())
    bias = (0.5 - s[0]).float()                                # row 0: every other choice is 0.5 up to rounding
    bias[[50, 9]] = INF
    for k in (1, 2, 3, 8):
        check_route(x, k, bias, score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,best,forced", [(64, 8, 2, [5]), (64, 8, 2, [5, 60, 61, 17]), (64, 8, 1, [40, 41, 42]), (60, 5, 2, [59]),
                                                  (512, 32, 2, [100, 200, 300, 301]), (30, 2, 2, [0, 29])])
def test_groups_of_an_expert_with_an_infinite_bias(E, groups, best, forced, score):
    """Their groups come first, ties of groups to the lower index, whether or
    not the other groups are too close for FP32."""
    g = torch.Generator().manual_seed(E + groups)
    x = logits_of(40, E, torch.float32, E)
    near = logits_of(1, E // groups, torch.float32, 4)[0].repeat(groups)[None].repeat(20, 1)
    near = near + torch.randint(-2, 3, near.shape, generator=g).float() * 2.0 ** -23 * near.abs()
    x = torch.cat([x, near])
    x[1, forced] = -INF
    bias = torch.zeros(E)
    bias[forced] = INF
    for top in {1, max(1, groups // 2), groups - 1, groups}:
        for k in (1, 3):
            check_route(x, k, bias, score=score, n_groups=groups, top_groups=top, group_best=best)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("groups", [1, 8])
@pytest.mark.parametrize("biased", [False, True])
def test_logits_of_plus_infinity(biased, groups, renormalize, score, dtype):
    """Chosen like the largest finite value; a softmax over one is NaN, and its
    weights say so in every mode; other rows and sigmoids are as ever."""
    T, E, k = 24, 64, 5
    x = logits_of(T, E, dtype, 31)
    x[0, 7] = INF
    x[1, [3, 50, 51]] = INF
    x[2] = INF
    x[3, 9] = INF
    x[3, 10:] = -INF
    x[4, 20] = INF
    x[4, 21] = float("nan")
    x[5, 30] = INF
    x[5, :30] = torch.finfo(dtype).min
    x[6, 40] = INF                                             # an expert that its bias masks
    bias = (torch.rand(E, generator=torch.Generator().manual_seed(2)) - 0.5) * 0.2
    if biased:
        bias[40] = -INF
    kw = dict(score=score, renormalize=renormalize, n_groups=groups, top_groups=max(1, groups // 2))
    w, ids = dg.det_moe_route(x.cuda(), k, bias=bias.cuda() if biased else None, **kw)
    ok()
    large = ref.f64(x)
    large[large == INF] = np.finfo(np.float32).max
    rw, rids = ref.route(large, k, bias=ref.f64(bias) if biased else None, **kw)
    assert np.array_equal(ids.cpu().numpy(), rids)
    w = ref.f64(w)
    inf = (ref.f64(x) == INF).any(1) if score == "softmax" else np.zeros(T, dtype=bool)
    assert np.isnan(w[inf][rids[inf] >= 0]).all() and not w[inf][rids[inf] < 0].any()
    assert (np.abs(w - rw)[~inf] <= np.abs(rw[~inf]) * (2 * 20 + 64) * 2.0 ** -24 + 1e-37).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("low,groups,top,k", [([1], 2, 2, 10), ([0], 2, 2, 12), ([1, 2], 3, 2, 12), ([0, 1, 2, 3], 4, 2, 9), ([5, 6], 8, 7, 32)])
def test_groups_whose_biases_are_the_lowest_finite_value(low, groups, top, k, score, dtype):
    """Their values are below FP32's range, and they are groups all the same."""
    E, size = groups * 8, 8
    x = logits_of(20, E, dtype, 8 + groups)
    bias = torch.zeros(E)
    for h in low:                                              # equal logits: exact ties, to the lower index
        bias[h * size:(h + 1) * size] = torch.finfo(torch.float32).min
        x[:, h * size:(h + 1) * size] = 0.5
    check_route(x, k, bias, score=score, n_groups=groups, top_groups=top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("large", [64.0, 1024.0])
def test_a_group_whose_large_biases_cancel(large, score):
    """Groups of two whose values FP32 tells apart, and one with biases of both
    signs, whose value is as small and whose error is not: wherever it comes
    among them, the kept groups are those of 64 bits."""
    T, G = 60, 8
    g = torch.Generator().manual_seed(int(large))
    for t in range(T):
        value = 0.1 + 2e-5 * torch.randperm(G, generator=g).double()
        first = value * (0.3 + 0.4 * torch.rand(G, generator=g, dtype=torch.float64))
        s = torch.stack([first, value - first], 1)
        h = t % (G - 1)
        bias = torch.zeros(G, 2)
        bias[h] = torch.tensor([large, -large])
        if score == "softmax":                                 # the last group takes what is left, and no part
            s[-1] = (1.0 - s[:-1].sum()) / 2
            bias[-1] = -INF
            x = torch.log(s)
        else:
            x = torch.log(s / (1.0 - s))
        x = x.reshape(1, 2 * G).float()
        for top in range(1, G - 1):
            check_route(x, 2, bias.reshape(-1), score=score, n_groups=G, top_groups=top)


@pytest.mark.parametrize("far", [60.0, 85.0, 95.0, 102.0])
@pytest.mark.parametrize("shift", [0.0, 0.37])
def test_scores_far_below_the_rows_largest(far, shift):
    """Choices among softmax scores of 1e-26 to below FP32's normal numbers, whose
    logits are a few units in the last place apart: the argument's rounding alone
    is as large. Biases of zero leave the logits' order."""
    T, E = 100, 64
    g = torch.Generator().manual_seed(int(far))
    x = torch.full((T, E), -far) - torch.randint(0, 200, (T, E), generator=g).float() * 2.0 ** -17
    x[:, 5] = 0.0
    x = x + shift * torch.rand((T, 1), generator=g)
    for k in (2, 8, 20):
        check_route(x, k, torch.zeros(E))
        check_route(x, k, torch.zeros(E), n_groups=4, top_groups=2)
