"""A mixture-of-experts language-model block on the package's operators.

One block: embedding, RMSNorm, router, experts (two 8-bit products around a
squared ReLU), residual, LM head. ``train_step`` runs it forward and backward
and returns the loss and every gradient; ``forward`` alone is what serving
runs. Everything but the element-wise glue is a det_* operator, so the
block inherits their guarantees, and ``main`` shows both:

  - a token's logits are the same bits alone, in a batch, and in any batch;
  - a training step gives the same bits every time.

    python examples/moe_block.py [--tokens 2048] [--hidden 1024] ...
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import invariant_deterministic_gemm_gb300 as dg  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


def pitched(x):
    """x with rows that begin on 16 bytes, as the BF16 products want them."""
    n = x.shape[1]
    out = x.new_zeros((x.shape[0], -(-n // 8) * 8))
    out[:, :n] = x
    return out[:, :n]


class Block:
    """The block's weights: BF16 masters, and the experts' 8-bit copies."""

    def __init__(self, vocab, hidden, ffn, experts, top_k, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def randn(*shape, std=0.02):
            return (torch.randn(shape, generator=g, device="cuda") * std).to(BF16)

        self.vocab, self.hidden, self.experts, self.top_k = vocab, hidden, experts, top_k
        self.scale = math.sqrt(hidden)
        self.table = randn(vocab, hidden)
        self.norm = torch.ones(hidden, dtype=BF16, device="cuda")
        self.router = randn(experts, hidden)
        self.bias = torch.zeros(experts, device="cuda")       # balance bias: moves the choice, not the weights
        self.up = randn(experts, ffn, hidden)
        self.down = randn(experts, hidden, ffn)
        self.head = randn(vocab, hidden)
        self.eps = 1e-6
        self.quantize()

    def quantize(self):
        """The experts' 8-bit weights, as they lie and transposed (for the input
        gradients); once after every update of the masters."""
        self.up_q, self.down_q = dg.det_fp8_quantize_tiles(self.up), dg.det_fp8_quantize_tiles(self.down)
        self.up_t = dg.det_fp8_quantize_tiles(self.up, transposed=True)
        self.down_t = dg.det_fp8_quantize_tiles(self.down, transposed=True)

    def route_args(self):
        return dict(score="sigmoid", renormalize=True, scale=1.0)

    def forward(self, tokens, keep=None):
        """Logits [T, vocab] FP32; keep (a dict) receives what the backward pass needs."""
        h0 = dg.det_embedding(tokens, self.table, self.scale)
        hn = dg.det_rmsnorm(h0, self.norm, self.eps)
        scores = dg.det_gemm_fwd_fp32_rhs_transposed(hn, self.router)
        w, ids = dg.det_moe_route(scores, self.top_k, bias=self.bias, **self.route_args())
        offsets, rows, slots = dg.det_moe_dispatch(ids, self.experts)
        xq, xs = dg.det_fp8_quantize_rows(hn, rows, self.top_k)          # gather and quantise
        up = dg.det_fp8_gemm_grouped(xq, xs, *self.up_q, offsets)
        act = torch.relu(up).square()
        ys = dg.det_fp8_gemm_grouped(*dg.det_fp8_quantize_rows(act), *self.down_q, offsets)
        h1 = h0 + dg.det_moe_combine(ys, slots, w)
        logits = dg.det_gemm_fwd_fp32_rhs_transposed(h1, self.head)
        if keep is not None:
            keep.update(h0=h0, hn=hn, scores=scores, w=w, ids=ids, offsets=offsets, rows=rows, slots=slots, up=up, act=act,
                        ys=ys, h1=h1)
        return logits

    def train_step(self, tokens, targets):
        """(loss, gradients by name) of the mean cross entropy."""
        s = {}
        logits = self.forward(tokens, s)
        T = tokens.shape[0]
        logp = torch.log_softmax(logits, 1)
        loss = -logp.gather(1, targets[:, None]).mean()
        p = logp.exp()
        p[torch.arange(T, device="cuda"), targets] -= 1.0
        dlogits = (p / T).to(BF16)
        g = {"head": dg.det_gemm_db_transposed(s["h1"], dlogits)}
        dh1 = dg.det_gemm_fwd(dlogits, self.head)
        # experts
        off = s["offsets"]
        dys, dw = dg.det_moe_combine_bwd(dh1, s["ys"], s["rows"], s["slots"], s["w"])
        dact = dg.det_fp8_gemm_grouped(*dg.det_fp8_quantize_rows(dys), *self.down_t, off)
        g["down"] = dg.det_fp8_gemm_wgrad(*dg.det_fp8_quantize_cols(dys, off), *dg.det_fp8_quantize_cols(s["act"], off), off)
        dup = dact * (2.0 * torch.relu(s["up"]))
        dxs = dg.det_fp8_gemm_grouped(*dg.det_fp8_quantize_rows(dup), *self.up_t, off)
        xs = dg.det_moe_gather(s["hn"], s["rows"], self.top_k)
        g["up"] = dg.det_fp8_gemm_wgrad(*dg.det_fp8_quantize_cols(dup, off), *dg.det_fp8_quantize_cols(xs, off), off)
        dhn = dg.det_moe_combine(dxs, s["slots"]).float()
        # router
        dscores = dg.det_moe_route_bwd(dw, s["scores"], s["ids"], **self.route_args())
        dscores = pitched(dscores.to(BF16))
        g["router"] = dg.det_gemm_db_transposed(s["hn"], dscores)
        dhn += dg.det_gemm_fwd(dscores, self.router).float()
        # RMSNorm: y = x r w, r = 1 / sqrt(mean x^2 + eps)
        x = s["h0"].float()
        r = torch.rsqrt(x.square().mean(1, keepdim=True) + self.eps)
        g["norm"] = (dhn * x * r).sum(0)
        dx = dhn * self.norm.float()
        dh0 = dh1.float() + r * (dx - x * (r * r) * (dx * x).mean(1, keepdim=True))
        g["table"] = dg.det_embedding_grad(dh0.to(BF16), tokens, self.vocab, self.scale)
        return loss, g


def main(argv=None):
    a = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    a.add_argument("--tokens", type=int, default=2048)
    a.add_argument("--vocab", type=int, default=16384)
    a.add_argument("--hidden", type=int, default=1024)
    a.add_argument("--ffn", type=int, default=1792)
    a.add_argument("--experts", type=int, default=8)
    a.add_argument("--top-k", type=int, default=2)
    a.add_argument("--steps", type=int, default=3)
    a.add_argument("--lr", type=float, default=1e-3)
    o = a.parse_args(argv)
    block = Block(o.vocab, o.hidden, o.ffn, o.experts, o.top_k)
    g = torch.Generator(device="cuda").manual_seed(1)
    tokens = torch.randint(0, o.vocab, (o.tokens,), generator=g, device="cuda")
    targets = torch.roll(tokens, -1)

    logits = block.forward(tokens)
    alone = all(torch.equal(block.forward(tokens[t:t + n]), logits[t:t + n])
                for t, n in ((0, 1), (o.tokens - 1, 1), (o.tokens // 2, min(33, o.tokens - o.tokens // 2))))
    first, again = block.train_step(tokens, targets), block.train_step(tokens, targets)
    same = torch.equal(first[0], again[0]) and all(torch.equal(first[1][k], again[1][k]) for k in first[1])
    losses = []
    for _ in range(o.steps):
        loss, grads = block.train_step(tokens, targets)
        losses.append(float(loss))
        for name, d in grads.items():
            w, d = getattr(block, name), d.float()
            w.copy_(w.float() - o.lr * d / (d.square().mean().sqrt() + 1e-12))
        block.quantize()
    assert dg.det_gemm_check() == 0
    print("logits of a token alone and in the batch: %s" % ("the same bits" if alone else "DIFFERENT"))
    print("gradients of two runs: %s" % ("the same bits" if same else "DIFFERENT"))
    print("loss: " + " -> ".join("%.4f" % v for v in losses))
    return alone, same, losses


if __name__ == "__main__":
    main()
