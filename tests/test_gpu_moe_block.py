"""The example block runs its operators together as a program does: a token's
logits do not depend on its batch, a training step repeats bit for bit, a few
steps lower the loss, and its gradients agree with 64-bit differences of a
plain FP32 model to the 8-bit operands' accuracy."""
import os
import sys

import pytest
import torch

import invariant_deterministic_gemm_gb300 as dg

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_the_block_is_batch_invariant_and_repeatable_and_learns():
    import moe_block
    alone, same, losses = moe_block.main(["--tokens", "257", "--vocab", "2048", "--hidden", "264", "--ffn", "200", "--experts", "6",
                                          "--top-k", "2", "--steps", "4"])
    assert alone and same
    assert losses[-1] < losses[0]


def test_the_blocks_gradients_point_where_a_plain_model_goes():
    """Cosine between each gradient and autograd's of the same block in FP32
    with unquantised weights. An e4m3 rounding is off by at most 2^-4 of a
    value (about 2^-5.8 in the mean square), each expert product has two such
    operands, and a gradient passes at most four of them: relative errors
    of about sqrt(8) 2^-5.8 = 0.05, so cosines above 1 - 0.05^2 = 0.9975; half
    of that distance again is left for BF16 roundings."""
    import moe_block
    T, V, H, F, E, k = 192, 512, 256, 384, 4, 2
    block = moe_block.Block(V, H, F, E, k, seed=3)
    g = torch.Generator(device="cuda").manual_seed(5)
    tokens = torch.randint(0, V, (T,), generator=g, device="cuda")
    targets = torch.roll(tokens, -1)
    keep = {}
    block.forward(tokens, keep)
    loss, grads = block.train_step(tokens, targets)
    p = {n: getattr(block, n).float().clone().requires_grad_() for n in grads}
    h0 = p["table"][tokens] * block.scale
    hn = h0 * torch.rsqrt(h0.square().mean(1, keepdim=True) + block.eps) * p["norm"]
    s = torch.sigmoid(hn @ p["router"].T)
    ids = keep["ids"].long()                                    # the choice is held fixed
    w = s.gather(1, ids)
    w = w / (w.sum(1, keepdim=True) + 1e-20)
    y = torch.zeros_like(h0)
    for e in range(E):
        ye = torch.relu(hn @ p["up"][e].T).square() @ p["down"][e].T
        y = y + ye * ((ids == e) * w).sum(1, keepdim=True)
    want = torch.nn.functional.cross_entropy((h0 + y) @ p["head"].T, targets)
    want.backward()
    assert abs(float(loss) - float(want)) < 0.01 * float(want)
    for n, d in grads.items():
        a, b = d.double().flatten(), p[n].grad.double().flatten()
        cos = float(a @ b / (a.norm() * b.norm()))
        assert cos > 0.996, (n, cos)
    assert dg.det_gemm_check() == 0
