"""GPU parity of the MoE routing operators against the float64 oracle: layouts
and counts exactly; losses and gradients within bounds from their definitions.

A score is exp(u - max) / sum in fp32: the exponent's argument (at most ~100
in size here) is rounded to 2^-24 of its size and the hardware exp2, log2 and
the division are good to a few units, so a score is within 2^-16 of its value
for |u| < 100 (2^-19 for |u| < 10). A loss is a sum of positive terms in such
scores; a gradient is g s (w - s.w), off by at most that share of g s (|w| +
s.|w|). bf16 gradients add 2^-8 of their value.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fine_grained_fp8_quantize_amd as fq
from oracle import moe

pytestmark = pytest.mark.gpu


def routes(seed, tokens, topk, experts, lost=0.1):
    rng = np.random.default_rng([seed, tokens, experts])
    ids = np.argsort(rng.random((tokens, experts)) - 0.4 * (np.arange(experts) % 3 == 0), axis=1)[:, :topk]
    ids = np.concatenate([ids, np.full((tokens, topk - ids.shape[1]), -1)], axis=1)
    return np.where(rng.random(ids.shape) < lost, rng.integers(-3, 0, ids.shape), ids).astype(np.int32)


@pytest.mark.parametrize("tokens,topk,experts,first,align", [
    (1, 1, 1, 0, 1), (1, 8, 8, 0, 16), (63, 1, 2, 0, 128), (64, 3, 5, 2, 16), (65, 8, 64, 0, 128), (1000, 8, 256, 0, 16),
    (1024, 8, 33, 100, 128), (1025, 8, 32, 0, 16), (5000, 4, 7, 0, 1), (20000, 8, 256, 32, 128), (3000, 6, 1024, 0, 16)])
def test_dispatch(tokens, topk, experts, first, align):
    ids = routes(1, tokens, topk, first + experts + 5)
    off, rows, dst = fq.moe_dispatch(torch.from_numpy(ids).cuda(), experts, align, first)
    want = moe.dispatch(ids, experts, align, first)
    for got, ref, name in zip((off, rows, dst), want, ("offsets", "rows", "destinations")):
        assert np.array_equal(got.cpu().numpy(), ref), name


@pytest.mark.parametrize("tokens", [700, 9000])
def test_dispatch_one_sided(tokens):
    """Every route to one expert, to none, and repeated ids in a token."""
    for ids in (np.full((tokens, 4), 3), np.full((tokens, 4), -1), np.tile([2, 2, 0, 2], (tokens, 1))):
        ids = ids.astype(np.int32)
        got = fq.moe_dispatch(torch.from_numpy(ids).cuda(), 5, 16)
        for g, ref in zip(got, moe.dispatch(ids, 5, 16, 0)):
            assert np.array_equal(g.cpu().numpy(), ref)


def test_dispatch_without_tokens():
    off, rows, dst = fq.moe_dispatch(torch.empty((0, 4), dtype=torch.int32, device="cuda"), 6, 16)
    assert off.tolist() == [0] * 7 and rows.tolist() == [0] * 6 and dst.shape == (0, 4)


def cuts(rng, tokens, seqs):
    return np.concatenate([[0], np.sort(rng.integers(0, tokens + 1, seqs - 1)), [tokens]]).astype(np.int32)


def balance_case(x, ids, offsets, score, dtype, share, grad=1.25, alpha=0.5, strided=False):
    logits = torch.from_numpy(x).to(dtype).cuda()
    x = logits.double().cpu().numpy()
    if strided:
        big = torch.full((x.shape[0], x.shape[1] + 3), float("nan"), dtype=dtype, device="cuda")
        big[:, :x.shape[1]] = logits
        logits = big[:, :x.shape[1]]
    d_ids = torch.from_numpy(ids).cuda()
    d_off = None if offsets is None else torch.from_numpy(offsets).cuda()
    off = [0, len(x)] if offsets is None else offsets
    loss, counts, coef = fq.moe_balance_loss(logits, d_ids, d_off, score, alpha)
    want, n, w = moe.balance(x, ids, off, score, alpha)
    assert np.array_equal(counts.cpu().numpy(), n)
    assert np.allclose(coef.double().cpu().numpy(), w, rtol=2.0 ** -20, atol=0)
    assert float(loss) == pytest.approx(want, rel=share + 2.0 ** -18, abs=0)
    g = torch.tensor([grad], device="cuda")
    out = torch.full(logits.shape, 9.0, dtype=dtype, device="cuda")
    d = fq.moe_balance_loss_backward(logits, d_ids, coef, g, d_off, score, out=out).double().cpu().numpy()
    ref = moe.balance_gradient(x, ids, off, score, w, grad)
    s = moe.scores(x, score)
    seq = np.searchsorted(np.asarray(off)[1:], np.arange(len(x)), side="right")
    tol = (2 * share + 2.0 ** -18) * grad * s * (w[seq] + (s * w[seq]).sum(1, keepdims=True)) + 1e-37
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol) + 1e-37
    assert (np.abs(d - ref) <= tol).all()
    return loss, counts, coef


@pytest.mark.parametrize("tokens,experts,topk,seqs", [
    (1, 1, 1, 1), (1, 8, 2, 3), (3, 64, 8, 2), (63, 65, 1, 1), (64, 128, 4, 2), (65, 129, 8, 4), (200, 256, 8, 9),
    (300, 20, 3, 70), (1000, 1000, 8, 3), (129, 257, 2, 2), (2500, 513, 2, 5)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_balance(tokens, experts, topk, seqs, score, dtype):
    rng = np.random.default_rng([tokens, experts])
    x = (2 * rng.standard_normal((tokens, experts)) - 0.3).astype(np.float32)
    ids = routes(2, tokens, topk, experts)
    ids[rng.random(tokens) < 0.1] = -1
    balance_case(x, ids, cuts(rng, tokens, seqs) if seqs > 1 else None, score, dtype, 2.0 ** -19)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_long_batch(score):
    """More tokens than parts of 64."""
    rng = np.random.default_rng(8)
    x = rng.standard_normal((70000, 16)).astype(np.float32)
    balance_case(x, routes(3, 70000, 2, 16), np.array([0, 100, 65000, 70000], np.int32), score, torch.float32, 2.0 ** -19)


def test_balance_many_sequences():
    """As many sequences as there may be, most of a token or none (a lane adds
    up to 512 of their losses, one after the other)."""
    rng = np.random.default_rng(12)
    x = rng.standard_normal((40000, 8)).astype(np.float32)
    ids = routes(9, 40000, 2, 8)
    ids[rng.random(40000) < 0.3] = -1
    balance_case(x, ids, cuts(rng, 40000, 32768), "softmax", torch.float32, 2.0 ** -14)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_masked_and_extreme_logits(score):
    rng = np.random.default_rng(9)
    x = (rng.standard_normal((40, 70)) * 20).astype(np.float32)
    x[:, 5] = -np.inf                       # an expert that is switched off
    x[3] = -np.inf                          # nothing left in the row
    x[4] = np.finfo(np.float32).min         # the lowest value everywhere
    x[5, 1:] = np.finfo(np.float32).min
    x[6] = -95.0 + x[6] / 50                # sigmoids that underflow
    x[7] = 90.0 + x[7] / 50                 # sigmoids of one
    x[7, 5] = -np.inf
    x[6, 5] = -np.inf
    balance_case(x, routes(4, 40, 4, 70, 0.0), None, score, torch.float32, 2.0 ** -16, strided=True)


def test_balance_uncounted_rows_do_not_matter():
    x = np.zeros((10, 8), np.float32)
    x[4] = np.nan
    ids = routes(5, 10, 2, 8, 0.0)
    ids[4] = -1
    balance_case(np.where(np.isnan(x), 7.0, x), ids, None, "softmax", torch.float32, 2.0 ** -19)
    d_ids, logits = torch.from_numpy(ids).cuda(), torch.from_numpy(x).cuda()
    loss, _, coef = fq.moe_balance_loss(logits, d_ids)
    assert torch.isfinite(loss).all()
    d = fq.moe_balance_loss_backward(logits, d_ids, coef)
    assert torch.isfinite(d).all() and (d[4] == 0).all()
    ids[4, 0] = 1                            # now it counts
    loss, _, coef = fq.moe_balance_loss(logits, torch.from_numpy(ids).cuda())
    assert torch.isnan(loss).all()


def test_balance_without_tokens_or_routes():
    none = torch.empty((0, 8), device="cuda")
    loss, counts, coef = fq.moe_balance_loss(none, torch.empty((0, 2), dtype=torch.int32, device="cuda"))
    assert float(loss) == 0 and (counts == 0).all() and (coef == 0).all()
    x = torch.randn((30, 8), device="cuda")
    ids = torch.full((30, 2), -1, dtype=torch.int32, device="cuda")
    loss, counts, coef = fq.moe_balance_loss(x, ids)
    assert float(loss) == 0 and (counts == 0).all() and (coef == 0).all()
    assert (fq.moe_balance_loss_backward(x, ids, coef) == 0).all()


def test_balance_gradient_against_differences():
    """The kernel's gradient against central differences of the kernel's loss."""
    torch.manual_seed(0)
    x = torch.randn((6, 5), device="cuda")
    ids = torch.from_numpy(routes(6, 6, 2, 5, 0.0)).cuda()
    for score in ("softmax", "sigmoid"):
        _, _, coef = fq.moe_balance_loss(x, ids, None, score)
        d = fq.moe_balance_loss_backward(x, ids, coef, None, None, score)
        h = 2.0 ** -7
        for t in range(6):
            for e in range(5):
                hi, lo = x.clone(), x.clone()
                hi[t, e] += h
                lo[t, e] -= h
                diff = (float(fq.moe_balance_loss(hi, ids, None, score)[0])
                        - float(fq.moe_balance_loss(lo, ids, None, score)[0])) / (2 * h)
                # third derivatives (below 2) times h^2 / 6, and the losses' rounding over 2 h
                assert abs(float(d[t, e]) - diff) < 2 * h * h / 6 + 2.0 ** -19 * 2 / (2 * h)


def test_balance_repeats_bit_for_bit_in_place_and_on_another_stream():
    rng = np.random.default_rng(10)
    x = torch.from_numpy(rng.standard_normal((3000, 200)).astype(np.float32)).cuda()
    ids = torch.from_numpy(routes(7, 3000, 6, 200)).cuda()
    first = fq.moe_balance_loss(x, ids)
    d = fq.moe_balance_loss_backward(x, ids, first[2])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        again = fq.moe_balance_loss(x, ids, stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    y = x.clone()
    assert fq.moe_balance_loss_backward(y, ids, first[2], out=y) is y and torch.equal(y, d)
