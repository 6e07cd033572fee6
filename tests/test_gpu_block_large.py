"""Sizes past 32 bits: the optimizer, the gated products, their gradients and
the weight-only products over arrays of more than 2^32 bytes or elements. A
part of the result is compared with the same call on that part alone, or with
the CPU model."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fine_grained_fp8_quantize_amd as fq
from oracle import adamw as model

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def _free():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def test_optimizer_past_32_bits_of_elements():
    n, tail = (1 << 32) + 700, 3000  # (the tail crosses 2^32)
    f = lambda dt: torch.zeros(n, dtype=dt, device="cuda")  # noqa: E731
    p, g, m, v = f(torch.bfloat16), f(torch.bfloat16), f(torch.uint8), f(torch.uint8)
    s = [torch.zeros(-(-n // 128), device="cuda") for _ in range(2)]
    rng = np.random.default_rng(1)
    h = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
    pv, gv = ((model.bf16(rng.standard_normal(tail).astype(np.float32)).astype(np.uint32) << 16).view(np.float32)
              for _ in range(2))
    first = n - tail
    p[first:], g[first:] = torch.from_numpy(pv).cuda(), torch.from_numpy(gv).cuda()
    fq.adamw_step(fq.adamw_plan([p], [m], [v], [s[0]], [s[1]]), [g], 3, seed=11, **h)
    zero = np.zeros(tail, np.float32)
    want, mm, rr, _ = model.step32(pv, gv, zero, zero, step=3, **h)
    got = p[first:].view(torch.int16).cpu().numpy()
    assert np.array_equal(got, model.bf16(want).view(np.int16))
    assert not p[:first].any() and not m[:first].any()
    # whole blocks, on either side of 2^32
    cut = -first % 128
    for at, end in ((first + cut, 1 << 32), (1 << 32, n)):
        part = slice(at - first, end - first)
        bits = model.random_bits(end - at, 0, 3, 11, at)
        for codes, scales, x, half, root in ((m, s[0], mm, bits & np.uint64(0xFFFF), False),
                                             (v, s[1], rr, bits >> np.uint64(16), True)):
            c, sc = model.encode(x[part], half, root)
            assert np.array_equal(codes[at:end].cpu().numpy(), c)
            assert np.array_equal(scales[at // 128:-(-end // 128)].cpu().numpy(), sc)


@pytest.mark.parametrize("m", [3, 2200])
def test_gated_products_of_weights_past_32_bits(m):
    n, k = 131072 * 5, 7168  # 4.7 GB each
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    b = torch.randint(0, 0x70, (2, n, k), dtype=torch.uint8, device="cuda", generator=g)
    bs = torch.rand((2, n // 128, k // 128), device="cuda", generator=g) / 4096
    a = torch.randint(0, 0x70, (m, k), dtype=torch.uint8, device="cuda", generator=g)
    a_s = torch.rand((k // 128, m), device="cuda", generator=g) / 64
    out = fq.fp8_gated_gemm(a, a_s, b, bs)
    at = n - 256
    part = fq.fp8_gated_gemm(a, a_s, b[:, at:], bs[:, at // 128:])
    if m <= 64:
        assert torch.equal(out[:, at:], part)
    else:  # the part takes the rows kernel: other orders of the same sums, two roundings to bf16
        x, y = out[:, at:].double(), part.double()
        assert torch.all((x - y).abs() <= 2.0 ** -7 * y.abs() + 1e-3 * y.square().mean().sqrt())


@pytest.mark.parametrize("transposed", [False, True])
def test_gradients_past_32_bits(transposed):
    n = 2048
    m = (1 << 31) // n + 1024  # 2^31 elements and more of H: 2^32 of gate and up
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    dh = torch.empty((m, n), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    gu = torch.empty((m, 2 * n), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    out = fq.fp8_gated_backward(dh, gu, transposed=transposed)
    at = m - 128
    part = fq.fp8_gated_backward(dh[at:], gu[at:], transposed=transposed)
    assert torch.equal(out[0][at:].view(torch.uint8), part[0].view(torch.uint8))
    assert torch.equal(out[1][:, at:], part[1])
    if transposed:
        assert torch.equal(out[2][:, at:].view(torch.uint8), part[2].view(torch.uint8))
        assert torch.equal(out[3][at // 128:], part[3])


@pytest.mark.parametrize("gated", [False, True])
def test_weight_only_products_past_32_bits(gated):
    n, k = 131072 * 10, 7168  # 4.7 GB of codes each
    q = torch.randint(0, 256, ((2,) if gated else ()) + (k // 128, n // 16, 1024), dtype=torch.uint8, device="cuda")
    s = torch.full(q.shape[:-3] + (k // 512, n // 16, 64), 0x78797A7B, dtype=torch.int32, device="cuda")
    x = torch.randn((3, k), device="cuda").to(torch.bfloat16)
    at = n - 160
    cut = (slice(None),) * (q.dim() - 2) + (slice(at // 16, None),)
    fn = fq.fp4_gated_gemv_mx if gated else fq.fp4_gemv_mx
    whole, part = fn(x, q, s, out_dtype=torch.float32), fn(x, q[cut], s[cut], out_dtype=torch.float32)
    # (other numbers of waves: other orders of the same sums)
    size = part.square().mean().sqrt()
    assert torch.all((whole[:, at:] - part).abs() <= 1e-5 * (part.abs() + size)) and torch.isfinite(whole).all()
