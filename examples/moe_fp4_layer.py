"""A mixture-of-experts layer on the FP4 operators, routing included.

    python examples/moe_fp4_layer.py [--tokens 512]

One step of an expert layer as a serving or training program runs it on one
GPU: router logits, top-k choice, the balance loss of the step with its
gradient, the expert-sorted row layout, tokens quantized to FP4 once and sent
to their experts' rows, the gate-and-up product of all experts, the activation,
the down product, and the weighted sum back into token order. The experts'
weights are quantized once, before the step. Nothing in the step waits for the
GPU: the layout's size is its upper bound.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import fine_grained_fp8_quantize_amd as fq  # noqa: E402

ALIGN = 16  # rows of an expert's segment: whole row tiles of the FP4 layout


class ExpertLayer:
    """``experts`` feed-forward networks (hidden -> 2 x inner -> hidden), their
    weights held in FP4."""

    def __init__(self, router: torch.Tensor, gate_up: torch.Tensor, down: torch.Tensor, topk: int):
        """``router`` fp32 [experts][hidden]; ``gate_up`` bf16 [experts][2 inner][hidden];
        ``down`` bf16 [experts][hidden][inner]."""
        self.router, self.topk = router, topk
        self.experts, self.hidden = router.shape
        self.inner = down.shape[2]
        self.gate_up = fq.fp4_quantize_mx(gate_up)
        self.down = fq.fp4_quantize_mx(down)

    def __call__(self, x: torch.Tensor, alpha: float = 0.01):
        """bf16 tokens [tokens][hidden] -> (bf16 output, balance loss, per-expert
        counts, gradient of the loss with respect to the router's logits)."""
        tokens = x.shape[0]
        logits = x.float() @ self.router.t()
        gates, ids = torch.topk(torch.softmax(logits, dim=1), self.topk, dim=1)
        gates = gates / gates.sum(dim=1, keepdim=True)
        ids = ids.int()

        loss, counts, coef = fq.moe_balance_loss(logits, ids, alpha=alpha)
        dlogits = fq.moe_balance_loss_backward(logits, ids, coef)

        offsets, rows, dst = fq.moe_dispatch(ids, self.experts, ALIGN)
        room = -(-(tokens * self.topk + self.experts * (ALIGN - 1)) // ALIGN) * ALIGN
        a = fq.fp4_quantize_mx_scatter(x, dst, room)
        h = fq.fp4_grouped_gemm_mx(offsets, rows, *a, *self.gate_up, 2 * self.inner)
        gate, up = h.float().split(self.inner, dim=1)
        act = (torch.nn.functional.silu(gate) * up).bfloat16()
        y = fq.fp4_grouped_gemm_mx(offsets, rows, *fq.fp4_quantize_mx(act), *self.down, self.hidden)
        out = (y[dst.long()].float() * gates.unsqueeze(2)).sum(dim=1).bfloat16()
        return out, loss, counts, dlogits


def random_layer(experts: int, hidden: int, inner: int, topk: int, seed: int = 0) -> ExpertLayer:
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda") * 0.02

    return ExpertLayer(normal(experts, hidden), normal(experts, 2 * inner, hidden).bfloat16(),
                       normal(experts, hidden, inner).bfloat16(), topk)


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--inner", type=int, default=1024)
    ap.add_argument("--topk", type=int, default=8)
    a = ap.parse_args()
    layer = random_layer(a.experts, a.hidden, a.inner, a.topk)
    x = torch.randn((a.tokens, a.hidden), device="cuda").bfloat16()
    for _ in range(3):
        out, loss, counts, _ = layer(x)
    torch.cuda.synchronize()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(10):
        layer(x)
    end.record()
    torch.cuda.synchronize()
    print("%d tokens, %d experts, top-%d: balance loss %.5f, rows per expert %d to %d, %.0f us a step" % (
        a.tokens, a.experts, a.topk, float(loss), int(counts.min()), int(counts.max()),
        start.elapsed_time(end) * 100))
    assert torch.isfinite(out).all()


if __name__ == "__main__":
    main()
