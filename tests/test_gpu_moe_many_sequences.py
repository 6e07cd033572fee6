"""The balance loss of as many sequences as there may be, most of whose losses
are small next to the first ones': none of them may be lost in the sum."""
from __future__ import annotations

import math

import pytest
import torch

import fine_grained_fp8_quantize_amd as fq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("experts", [64, 256])
def test_small_losses_behind_large_ones(experts):
    """One token per sequence, all to expert 0, whose score is 1 in the first 16
    sequences and 2^-25.5 in the others: sequence s has the loss experts * score /
    seqs. In a running FP32 sum every small term is below half a unit of the
    large one. Scores are good to 2^-19 at these logits, everything else in the
    sum to a few 2^-24; the small terms are 2^-14.5 of the loss together."""
    seqs, big, ratio = 32768, 16, 2.0 ** -25.5
    x = torch.zeros((seqs, experts), device="cuda")
    x[:, 0] = math.log(ratio / (1 - ratio) * (experts - 1))
    x[:big, 0] = 60.0
    ids = torch.zeros((seqs, 1), dtype=torch.int32, device="cuda")
    cuts = torch.arange(seqs + 1, dtype=torch.int32, device="cuda")
    loss, counts, _ = fq.moe_balance_loss(x, ids, cuts)
    assert (counts[:, 0] == 1).all() and (counts[:, 1:] == 0).all()
    score = torch.softmax(x.double(), dim=1)[:, 0]
    want = float(experts / seqs * score.sum())
    assert float(score[big:].sum() / score.sum()) > 2.0 ** -15
    assert abs(float(loss) / want - 1) < 2.0 ** -17
