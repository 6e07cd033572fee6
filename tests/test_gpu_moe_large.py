"""The balance loss and its gradient on a batch of more than 2^28 tokens, whose
gradient takes more than one launch: the ends of the batch against the same
operator on those rows alone, bit for bit."""
from __future__ import annotations

import pytest
import torch

import fine_grained_fp8_quantize_amd as fq

pytestmark = pytest.mark.gpu

TOKENS, EXPERTS = (1 << 28) + 1000, 2


def test_more_tokens_than_one_launch_takes():
    x = torch.zeros((TOKENS, EXPERTS), dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros((TOKENS, 1), dtype=torch.int32, device="cuda")
    ids[1::2] = 1
    ids[5::1024] = -1
    ids[-300:] = 0
    cut = torch.tensor([0, TOKENS - 700, TOKENS], dtype=torch.int32, device="cuda")
    spots = (0, (1 << 27) - 40, (1 << 28) - 40, TOKENS - 80)
    g = torch.Generator(device="cuda").manual_seed(0)
    for at in spots:
        x[at:at + 80] = torch.randn((80, EXPERTS), generator=g, device="cuda")
    loss, counts, coef = fq.moe_balance_loss(x, ids, cut)
    for e in range(EXPERTS):
        here = ids[:, 0] == e
        assert counts[0, e] == here[:TOKENS - 700].sum() and counts[1, e] == here[TOKENS - 700:].sum()
        del here
    d = fq.moe_balance_loss_backward(x, ids, coef, None, cut)
    for at in spots:
        for s in range(2):  # rows of each sequence, under that sequence's coefficients
            lo, hi = max(at, s * (TOKENS - 700)), min(at + 80, TOKENS - 700 if s == 0 else TOKENS)
            if lo < hi:
                want = fq.moe_balance_loss_backward(x[lo:hi], ids[lo:hi].contiguous(), coef[s:s + 1].contiguous())
                assert torch.equal(d[lo:hi], want), (at, s)
                assert (want != 0).any()
    # f sums to 2 over the experts and P is close to one half (all but a few logits are 0): close to 1
    assert abs(float(loss) - 1.0) < 2.0 ** -6
