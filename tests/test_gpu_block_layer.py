"""The operators of a gated feed-forward block together, as a program uses them:
training steps with FP32 master weights and 8-bit optimizer states, eager and
captured into a graph, and serving of the trained weights in FP4."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fine_grained_fp8_quantize_amd as fq
from oracle import gated as model

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
M, N, K = 256, 128, 384


class Block:
    """y = down(act(x Wg^T) * (x Wu^T)) with the gradients of both weights and an optimizer step."""

    def __init__(self, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.master = [torch.randn((2 * N, K), generator=g, device="cuda") * 0.06,
                       torch.randn((K, N), generator=g, device="cuda") * 0.09]
        self.w = [t.to(torch.bfloat16) for t in self.master]
        zeros = lambda dt: [torch.zeros(t.shape, dtype=dt, device="cuda") for t in self.master]  # noqa: E731
        scales = lambda: [torch.zeros(t.numel() // 128, device="cuda") for t in self.master]  # noqa: E731
        self.state = zeros(E4M3), zeros(E4M3), scales(), scales()
        self.plan = fq.adamw_plan(self.master, *self.state, self.w)
        self.step = torch.zeros(1, dtype=torch.int64, device="cuda")
        self.grads = [torch.empty(t.shape, device="cuda") for t in self.master]
        self.keep = torch.empty((M, 2 * N), dtype=torch.bfloat16, device="cuda")
        self.y = torch.empty((M, K), device="cuda")

    def train(self, x, dy):
        """One step for inputs x and the gradient dy of the output."""
        xq, xs = fq.fp8_quantize_act(x)
        wq, ws, wt, wts = fq.fp8_quantize_weight(self.w[0], transposed=True)
        dq, ds, dt, dts = fq.fp8_quantize_weight(self.w[1], transposed=True)
        h, hs = fq.fp8_gated_gemm(xq, xs, wq.view(2, N, K), ws.view(2, N // 128, K // 128), "silu", E4M3, gate_up=self.keep)
        fq.fp8_gemm(h, hs, dq, ds, "block", torch.float32, out=self.y)
        dyq, dys = fq.fp8_quantize_act(dy)
        dh = fq.fp8_gemm(dyq, dys, dt, dts, "block", torch.bfloat16)
        g, gs, gt, gts = fq.fp8_gated_backward(dh, self.keep, transposed=True)
        fq.fp8_gemm(g, gs, wt, wts, "block", torch.bfloat16)  # dX, for the layer below
        xt, xts = fq.fp8_quantize_act(x, "128x1")
        fq.fp8_gemm(gt, gts, xt, xts, "row", torch.float32, out=self.grads[0])
        dyt, dyts = fq.fp8_quantize_act(dy, "128x1")
        ht, hts = fq.fp8_retile_act_128x1(h, hs)
        fq.fp8_gemm(dyt, dyts, ht, hts, "row", torch.float32, out=self.grads[1])
        self.step.add_(1)
        fq.adamw_step(self.plan, self.grads, self.step, 1e-3, weight_decay=0.1, seed=5)

    def everything(self):
        return [*self.master, *self.w, *[t.view(torch.uint8) for ts in self.state[:2] for t in ts], *self.state[2],
                *self.state[3], self.keep, self.y, *self.grads]

    def serve(self, x):
        gate_up = fq.fp4_quantize_mx(self.w[0].view(2, N, K))
        down = fq.fp4_quantize_mx(self.w[1])
        return fq.fp4_gemv_mx(fq.fp4_gated_gemv_mx(x, *gate_up, N), *down, K, out_dtype=torch.float32), gate_up, down


def _inputs(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(100 + seed)
    return [(torch.randn((M, K), generator=g, device="cuda") * s).to(torch.bfloat16) for s in (1.0, 1e-2)]


def test_captured_training_is_eager_training():
    eager, other = Block(1), Block(1)
    x, dy = _inputs(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        other.train(x, dy)
    for step in range(4):
        a, b = _inputs(step)
        eager.train(a, b)
        x.copy_(a)
        dy.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for i, (p, q) in enumerate(zip(eager.everything(), other.everything())):
            assert torch.equal(p, q), (step, i)
    assert int(other.step) == 4


def test_gradients_and_update_of_a_step():
    """The weights' gradients against float64 on the same inputs: what lies between are roundings to E4M3 (2^-4 of
    each term) and bf16; then the masters move by about the rate in each element with a gradient."""
    block = Block(2)
    before = [t.clone() for t in block.master]
    w = [t.double().cpu().numpy() for t in block.w]
    x, dy = _inputs(7)
    block.train(x, dy)
    xv, dyv = x.double().cpu().numpy(), dy.double().cpu().numpy()
    gate, up = xv @ w[0][:N].T, xv @ w[0][N:].T
    h = model.act("silu", gate) * up
    d = np.concatenate(model.gradients("silu", dyv @ w[1], gate, up), 1)
    # four E4M3 operands on the way to dW of gate and up (x twice, W, down and dY in the gradient), three to dW of down
    for got, ref, terms in ((block.grads[0], d.T @ xv, 5), (block.grads[1], dyv.T @ h, 4), (block.y, h @ w[1].T, 4)):
        got = got.double().cpu().numpy()
        assert np.linalg.norm(got - ref) <= terms * 2.0 ** -4 * np.linalg.norm(ref)
    for t, b, g in zip(block.master, before, block.grads):
        moved = (t - b * (1 - 1e-4)).abs()
        # the first step: m / sqrt(v) is the gradient's sign, but for eps beside gradients near 1e-8
        assert torch.all(moved[g.abs() > 1e-5] <= 1.01e-3) and torch.all(moved[g.abs() > 1e-5] >= 0.99e-3)
    for t, c in zip(block.master, block.w):
        assert torch.equal(t.to(torch.bfloat16), c)


@pytest.mark.parametrize("tokens", [1, 5])
def test_serving_of_the_weights(tokens):
    block = Block(3)
    x = _inputs(1)[0][:tokens]
    y, gate_up, down = block.serve(x)
    v = [[fq.fp4_dequantize_mx(q[i], s[i], N, K, torch.float32).double().cpu().numpy() for i in (0, 1)]
         for q, s in (gate_up,)][0]
    dv = fq.fp4_dequantize_mx(*down, K, N, torch.float32).double().cpu().numpy()
    xv = x.double().cpu().numpy()
    h = model.act("silu", xv @ v[0].T) * (xv @ v[1].T)
    # H is rounded to bf16 between the two products
    room = 2.0 ** -8 * np.abs(h) @ np.abs(dv).T + 1e-5 * (np.abs(h) @ np.abs(dv).T + 1e-3)
    assert np.all(np.abs(y.double().cpu().numpy() - h @ dv.T) <= 1.01 * room)
