"""The FP4 and MoE operators together: the example layer against float64, the
step captured in a HIP graph, and the operators next to the FP8 path."""
from __future__ import annotations

import os
import sys

import numpy as np
import pytest
import torch

import fine_grained_fp8_quantize_amd as fq
import workloads as wl
from gpu_util import assert_grouped_close, dev_bf16, host_out
from oracle import fp4, moe

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_fp4_layer  # noqa: E402

pytestmark = pytest.mark.gpu


def bits(t: torch.Tensor) -> np.ndarray:
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def fp4_values(t: torch.Tensor) -> np.ndarray:
    v = bits(t)
    return fp4.values(*fp4.quantize(v.reshape(-1, v.shape[-1])))[:, :v.shape[-1]].reshape(v.shape)


def test_layer_against_float64():
    """Every token through its experts one by one, in float64 on the FP4
    values. The hidden activations are rounded to bf16 and then to FP4, so a
    last-bit difference of the fp32 sums can move an element by one FP4 code
    (a quarter of itself) where it lies on a rounding boundary: one element in
    some 2^5 at the most, of 96 in a sum, which leaves the norm of the output
    within 2 percent and a single output within 0.2 of its rms."""
    experts, hidden, inner, topk, tokens = 6, 192, 96, 2, 37
    g = torch.Generator(device="cuda").manual_seed(1)
    gate_up = (torch.randn((experts, 2 * inner, hidden), generator=g, device="cuda") * 0.1).bfloat16()
    down = (torch.randn((experts, hidden, inner), generator=g, device="cuda") * 0.1).bfloat16()
    router = torch.randn((experts, hidden), generator=g, device="cuda") * 0.1
    x = torch.randn((tokens, hidden), generator=g, device="cuda").bfloat16()
    out, loss, counts, dlogits = moe_fp4_layer.ExpertLayer(router, gate_up, down, topk)(x)
    logits = x.float() @ router.t()
    gates, ids = torch.topk(torch.softmax(logits, dim=1), topk, dim=1)
    gates = (gates / gates.sum(dim=1, keepdim=True)).double().cpu().numpy()
    ids = ids.cpu().numpy()
    xv, wv, dv = fp4_values(x), fp4_values(gate_up), fp4_values(down)
    ref = np.zeros((tokens, hidden))
    for t in range(tokens):
        for k in range(topk):
            e = ids[t, k]
            h = torch.from_numpy(wv[e] @ xv[t]).bfloat16().double().numpy()
            act = torch.from_numpy(h[:inner] / (1 + np.exp(-h[:inner])) * h[inner:]).bfloat16()
            ref[t] += gates[t, k] * (dv[e] @ fp4_values(act[None])[0])
    err = np.abs(out.double().cpu().numpy() - ref).max() / np.sqrt((ref ** 2).mean())
    assert err < 2e-1 and np.linalg.norm(out.double().cpu().numpy() - ref) < 2e-2 * np.linalg.norm(ref)
    want, n, w = moe.balance(logits.double().cpu().numpy(), ids, [0, tokens], "softmax", 0.01)
    assert np.array_equal(counts.cpu().numpy(), n) and float(loss) == pytest.approx(want, rel=1e-5)
    ref_d = moe.balance_gradient(logits.double().cpu().numpy(), ids, [0, tokens], "softmax", w, 1.0)
    assert np.allclose(dlogits.double().cpu().numpy(), ref_d, rtol=1e-3, atol=1e-5 * np.abs(ref_d).max())


@pytest.mark.parametrize("tokens", [3, 400])
def test_step_captured_in_a_graph(tokens):
    """Routing, loss, quantization and products captured once and replayed on
    new inputs: equal to the eager calls every time."""
    experts, hidden, inner, topk = 8, 256, 128, 2
    layer = moe_fp4_layer.random_layer(experts, hidden, inner, topk, seed=2)
    room = -(-(tokens * topk + experts * 15) // 16) * 16
    x = torch.zeros((tokens, hidden), device="cuda").bfloat16()
    logits = torch.zeros((tokens, experts), device="cuda")
    ids = torch.zeros((tokens, topk), dtype=torch.int32, device="cuda")

    def step():
        loss, counts, coef = fq.moe_balance_loss(logits, ids)
        d = fq.moe_balance_loss_backward(logits, ids, coef)
        off, rows, dst = fq.moe_dispatch(ids, experts, 16)
        h = fq.fp4_grouped_gemm_mx(off, rows, *fq.fp4_quantize_mx_scatter(x, dst, room), *layer.gate_up, 2 * inner)
        y = fq.fp4_gemm_mx(*fq.fp4_quantize_mx(x), *fq.fp4_quantize_mx(x), tokens, tokens, torch.float32)
        w = fq.fp4_gemm_mx(*fq.fp4_quantize_mx(x, "32x1"), *fq.fp4_quantize_mx(x, "32x1"), hidden, hidden, torch.float32)
        return loss, counts, d, off, rows, dst, h, y, w

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in range(4):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        logits.copy_(torch.randn(logits.shape, generator=g, device="cuda"))
        ids.copy_(torch.topk(logits, topk, dim=1).indices)
        graph.replay()
        torch.cuda.synchronize()
        eager = step()
        torch.cuda.synchronize()
        for a, b in zip(captured, eager):
            assert torch.equal(a, b)


def test_dispatch_feeds_the_fp8_path():
    """moe_dispatch's layout through fp8_quantize_act_scatter and fp8_grouped_gemm."""
    import oracle
    tokens, topk, experts, n, k = 200, 3, 4, 256, 256
    rng = np.random.default_rng(5)
    ids = np.argsort(rng.random((tokens, experts)), axis=1)[:, :topk].astype(np.int32)
    off, rows, dst = fq.moe_dispatch(torch.from_numpy(ids).cuda(), experts, 128)
    x, w = wl.activation(1, "tiny_fprop", 150, tokens, k, 50.0), np.stack(
        [wl.weight(1, "tiny_fprop", 151 + e, n, k) for e in range(experts)])
    m_total = int(off[-1])
    a, sa = fq.fp8_quantize_act_scatter(dev_bf16(x), dst, m_total)
    b, sb = fq.fp8_quantize_weight_grouped(dev_bf16(w.reshape(-1, k)).view(experts, n, k))
    c = fq.fp8_grouped_gemm(off, rows, a, sa, b, sb)
    o_off, o_rows, o_dst = moe.dispatch(ids, experts, 128, 0)
    ra, rs, _ = oracle.quant_act_scatter(x, o_dst.astype(np.int32), m_total)
    rb = [oracle.quant_weight_128x128(w[e]) for e in range(experts)]
    ref = oracle.grouped_gemm(o_off, o_rows, ra, rs, np.stack([r[0] for r in rb]), np.stack([r[1] for r in rb]))
    assert_grouped_close(host_out(c), ref, o_off, o_rows, "dispatched FP8 experts")
