"""Few bf16 rows times FP4 weights on the GPU, against float64 sums of the
values that the codes stand for: one row and many, odd sizes, pitches and
addresses, experts by ids, special values."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fine_grained_fp8_quantize_amd as fq
from oracle import gated as model

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _bf16(rng, *shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16).cuda()


def _weights(rng, *shape):
    """FP4 weights of bf16 [..][n][k], and their values in float64."""
    w = _bf16(rng, *shape, scale=0.05)
    flat = w.reshape(-1, *shape[-2:])
    q, s = fq.fp4_quantize_mx(flat)
    v = np.stack([fq.fp4_dequantize_mx(q[i], s[i], *shape[-2:], out_dtype=torch.float32).cpu().numpy()
                  for i in range(len(flat))]).astype(np.float64)
    lead = shape[:-2]
    return q.reshape(*lead, *q.shape[1:]), s.reshape(*lead, *s.shape[1:]), v.reshape(shape)


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _room(x, v, out):
    """The products are exact; a sum of K of them in any order is off by at most K U times the sum of magnitudes, and
    an output in bf16 by 2^-8 of itself."""
    return 1.01 * x.shape[-1] * U * (np.abs(x) @ np.abs(v).T) + (2.0 ** -8 * 1.001 * np.abs(out) if out is not None else 0)


SHAPES = [(1, 16, 32), (1, 2048, 512), (1, 130, 7168), (2, 7, 100), (5, 300, 129), (16, 64, 2048), (17, 50, 640),
          (33, 33, 1000), (64, 16, 256), (65, 40, 130), (200, 24, 384), (3, 1, 1), (4, 20, 8),
          (2, 5000, 200), (9, 9000, 640), (20, 5000, 264), (25, 8300, 512), (50, 4500, 392), (60, 8200, 640), (40, 9000, 1100), (48, 8300, 2000)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_products(m, n, k):
    rng = np.random.default_rng(m * 3 + n + k)
    x = _bf16(rng, m, k)
    q, s, v = _weights(rng, n, k)
    want = _np(x) @ v.T
    got = fq.fp4_gemv_mx(x, q, s, n, out_dtype=torch.float32)
    assert np.all(np.abs(_np(got) - want) <= _room(_np(x), v, None))
    assert torch.equal(fq.fp4_gemv_mx(x, q, s, n), got.to(torch.bfloat16))
    # rows on their own, at addresses of two bytes, from a pitch of their own into a pitch of their own
    buf = torch.full((m, k + 5), float("nan"), dtype=torch.bfloat16, device="cuda")
    buf[:, 1:k + 1] = x
    out = torch.full((m, n + 3), float("nan"), device="cuda")
    fq.fp4_gemv_mx(buf[:, 1:k + 1], q, s, n, out_dtype=torch.float32, out=out[:, 1:n + 1])
    assert torch.equal(out[:, 1:n + 1], got) and torch.isnan(out[:, 0]).all() and torch.isnan(out[:, n + 1:]).all()
    assert torch.equal(fq.fp4_gemv_mx(x[m // 2:m // 2 + 1], q, s, n, out_dtype=torch.float32), got[m // 2:m // 2 + 1])


def _gated_room(act, x, v):
    """h = act(g) u of two sums with their own rooms: the slope of either activation is at most 1.13, and the
    activation's own roundings, gelu's argument among them, stay below 512 U of it (|w| up to 88)."""
    g, u = x @ v[0].T, x @ v[1].T
    dg, du = _room(x, v[0], None), _room(x, v[1], None)
    a = model.act(act, g)
    return a * u, 1.13 * dg * (np.abs(u) + du) + np.abs(a) * du + 512 * U * np.abs(a * u) + 1e-30


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("m,n,k", [(1, 8, 32), (1, 2048, 640), (5, 41, 136), (16, 100, 2000), (20, 7, 256), (40, 24, 512),
                                   (70, 16, 1030)])
def test_gated(m, n, k, act):
    rng = np.random.default_rng(m + n)
    x = _bf16(rng, m, k)
    q, s, v = _weights(rng, 2, n, k)
    want, room = _gated_room(act, _np(x), v)
    got = fq.fp4_gated_gemv_mx(x, q, s, n, act, out_dtype=torch.float32)
    assert np.all(np.abs(_np(got) - want) <= room)
    assert torch.equal(fq.fp4_gated_gemv_mx(x, q, s, n, act), got.to(torch.bfloat16))


@pytest.mark.parametrize("tokens,topk,experts", [(1, 1, 1), (1, 8, 256), (16, 4, 32), (7, 3, 5), (40, 2, 3), (300, 3, 2),
                                                 (64, 32, 40), (128, 32, 1024)])
@pytest.mark.parametrize("own_rows", [False, True])
def test_experts(tokens, topk, experts, own_rows):
    """Experts that nobody chose, ids outside the range on both sides, one expert several times in a row of ids."""
    rng = np.random.default_rng(tokens + topk + experts)
    n, k, first = (24, 200, 10) if experts < 1024 else (10, 32, 10)
    ids = rng.integers(first - 3, first + experts + 3, (tokens, topk)).astype(np.int32)
    if tokens > 4:
        ids[1] = first
        ids[2] = -1
        ids[3] = np.array([-2 ** 31, 2 ** 31 - 1], np.int64).astype(np.int32)[rng.integers(0, 2, topk)]
    q, s, v = _weights(rng, experts, 2, n, k)
    x = _bf16(rng, *((tokens, topk, k) if own_rows else (tokens, k)))
    xv = _np(x) if own_rows else np.repeat(_np(x)[:, None], topk, 1)
    want, room = np.zeros((2, tokens, topk, n)), np.zeros((2, tokens, topk, n))
    for t in range(tokens):
        for j in range(topk):
            e = int(ids[t, j]) - first
            if 0 <= e < experts:
                row = xv[t, j][None]
                want[0, t, j], room[0, t, j] = row @ v[e, 0].T, _room(row, v[e, 0], None)
                want[1, t, j], room[1, t, j] = (a[0] for a in _gated_room("silu", row, v[e]))
    d = torch.from_numpy(ids).cuda()
    out = torch.full((tokens, topk, n + 8), float("nan"), device="cuda")
    fq.fp4_gemv_mx(x, q[:, 0], s[:, 0], n, d, first, torch.float32, out=out[..., :n])
    assert np.all(np.abs(_np(out[..., :n]) - want[0]) <= room[0]) and torch.isnan(out[..., n:]).all()
    got = fq.fp4_gated_gemv_mx(x, q, s, n, "silu", d, first, torch.float32)
    assert np.all(np.abs(_np(got) - want[1]) <= room[1])
    assert torch.equal(fq.fp4_gated_gemv_mx(x, q, s, n, "silu", d, first), got.to(torch.bfloat16))


@pytest.mark.parametrize("n", [16, 40, 2050])
def test_a_rank_without_experts(n):
    kt, rt = 2, -(-n // 16)
    x = torch.full((5, 256), float("nan"), dtype=torch.bfloat16, device="cuda")
    ids = torch.arange(15, dtype=torch.int32, device="cuda").reshape(5, 3) - 2
    for lead, f in (((0,), fq.fp4_gemv_mx), ((0, 2), fq.fp4_gated_gemv_mx)):
        q = torch.zeros((*lead, kt, rt, 1024), dtype=torch.uint8, device="cuda")
        s = torch.zeros((*lead, 1, rt, 64), dtype=torch.int32, device="cuda")
        out = torch.full((5, 3, n + 4), float("nan"), device="cuda")
        f(x, q, s, n, ids=ids, first=4, out_dtype=torch.float32, out=out[..., :n])
        assert (out[..., :n] == 0).all() and torch.isnan(out[..., n:]).all()


def test_special_values_stay_in_their_row_and_column():
    rng = np.random.default_rng(4)
    m, n, k = 5, 40, 300
    w, x = _bf16(rng, n, k), _bf16(rng, m, k)
    q, s = fq.fp4_quantize_mx(w)
    clean = fq.fp4_gemv_mx(x, q, s, n, out_dtype=torch.float32)
    w[7, 33], x[3, 5], x[4, 299] = float("nan"), float("inf"), float("nan")
    q, s = fq.fp4_quantize_mx(w)
    got = fq.fp4_gemv_mx(x, q, s, n, out_dtype=torch.float32)
    assert torch.isnan(got[:, 7]).all() and torch.isnan(got[4]).all() and not torch.isfinite(got[3]).any()
    keep = [j for j in range(n) if j != 7]
    assert torch.equal(got[:3, keep], clean[:3, keep])
    # what lies behind a row of x is not read: NaN there changes nothing
    buf = torch.full((3, 384), float("nan"), dtype=torch.bfloat16, device="cuda")
    buf[:, :k] = x[:3]
    assert torch.equal(fq.fp4_gemv_mx(buf[:, :k], q, s, n, out_dtype=torch.float32)[:, keep], clean[:3, keep])


def test_scales_over_the_whole_range():
    """Blocks of every exponent that bf16 values have. A row's sum is 36 * 2^e, past the largest FP32 value from e =
    123 on: an infinity there."""
    k = 32
    e = np.arange(-124, 125)
    w = np.ldexp(np.array([1.0, -3.0, 6.0, 0.5] * 8), 0)[None] * np.exp2(e.astype(np.float64))[:, None]
    wt = torch.from_numpy(w.astype(np.float32)).to(torch.bfloat16).cuda()
    q, s = fq.fp4_quantize_mx(wt)
    v = _np(fq.fp4_dequantize_mx(q, s, len(e), k, torch.float32))
    x = torch.ones((1, k), dtype=torch.bfloat16, device="cuda")
    got = _np(fq.fp4_gemv_mx(x, q, s, len(e), out_dtype=torch.float32))[0]
    want = v.sum(1)
    past = np.abs(want) > np.finfo(np.float32).max
    assert np.array_equal(past, e >= 123) and np.all(np.isposinf(got[past]))
    bad = np.flatnonzero(np.abs(got - want)[~past] > 32 * U * np.abs(v).sum(1)[~past])
    assert len(bad) == 0, (e[bad], got[bad], want[bad])


def test_pitched_and_interleaved_weights():
    """Gate and up rows of one [2n][k] matrix seen as two, and matrices with row tiles of others between theirs."""
    rng = np.random.default_rng(6)
    n, k = 48, 700
    w, x = _bf16(rng, 2 * n, k, scale=0.1), _bf16(rng, 3, k)
    q, s = fq.fp4_quantize_mx(w)
    v = _np(fq.fp4_dequantize_mx(q, s, 2 * n, k, torch.float32)).reshape(2, n, k)
    two = q.view(q.shape[0], 2, n // 16, 1024).permute(1, 0, 2, 3), s.view(s.shape[0], 2, n // 16, 64).permute(1, 0, 2, 3)
    want, room = _gated_room("silu", _np(x), v)
    got = fq.fp4_gated_gemv_mx(x, *two, n, out_dtype=torch.float32)
    assert np.all(np.abs(_np(got) - want) <= room)
    for i in (0, 1):
        y = fq.fp4_gemv_mx(x, two[0][i], two[1][i], n, out_dtype=torch.float32)
        assert np.all(np.abs(_np(y) - _np(x) @ v[i].T) <= _room(_np(x), v[i], None))


def test_empty_sizes():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    q, s = z(0, 2, 1024, dt=torch.uint8), z(0, 2, 64, dt=torch.int32)
    assert (fq.fp4_gemv_mx(z(3, 0), q, s, 20) == 0).all()
    assert (fq.fp4_gated_gemv_mx(z(3, 0), q[None].repeat(2, 1, 1, 1), s[None].repeat(2, 1, 1, 1), 20) == 0).all()
    q, s = fq.fp4_quantize_mx(z(20, 130))
    assert fq.fp4_gemv_mx(z(0, 130), q, s, 20).shape == (0, 20)
    ids = z(0, 4, dt=torch.int32)
    assert fq.fp4_gemv_mx(z(0, 130), q[None], s[None], 20, ids).shape == (0, 4, 20)


def test_streams_and_replays():
    rng = np.random.default_rng(8)
    q, s, _ = _weights(rng, 6, 2, 64, 512)
    xs = [_bf16(rng, 9, 512) for _ in range(2)]
    ids = torch.from_numpy(rng.integers(0, 7, (9, 2)).astype(np.int32)).cuda()
    want = [fq.fp4_gated_gemv_mx(x, q, s, 64, ids=ids) for x in xs]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], [torch.zeros_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(4):
        for i in (0, 1):
            fq.fp4_gated_gemv_mx(xs[i], q, s, 64, ids=ids, out=outs[i], stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    x, out, graph = xs[0].clone(), torch.zeros_like(want[0]), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fq.fp4_gated_gemv_mx(x, q, s, 64, ids=ids, out=out)
    for i in (1, 0, 1):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])


def test_refusals():
    rng = np.random.default_rng(9)
    q, s, _ = _weights(rng, 2, 40, 200)
    x, E = _bf16(rng, 3, 200), fq.Fp8qError
    ids = torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    bad = lambda match, fn, *a, **kw: pytest.raises(E, fn, *a, **kw).match(match)  # noqa: E731
    bad("x must be bfloat16", fq.fp4_gemv_mx, x.float(), q[0], s[0], 40)
    bad("K = 100", fq.fp4_gemv_mx, x[:, :100], q[0], s[0], 40)
    bad("does not fit", fq.fp4_gemv_mx, x, q[0], s[0], 60)
    bad("w must be uint8", fq.fp4_gemv_mx, x, q, s, 40)
    bad("w must be uint8", fq.fp4_gated_gemv_mx, x, q[0], s[0], 40)
    bad("w must be uint8", fq.fp4_gated_gemv_mx, x, q, s, 40, ids=ids)
    bad("stacked in twos", fq.fp4_gated_gemv_mx, x, q[:1], s[:1], 40)
    bad("act", fq.fp4_gated_gemv_mx, x, q, s, 40, "tanh")
    bad("w_scale", fq.fp4_gated_gemv_mx, x, q[None], s[None, :1], 40, ids=ids)
    bad("ids must be", fq.fp4_gemv_mx, x, q, s, 40, ids.long())
    bad("x must be \\[tokens\\]", fq.fp4_gemv_mx, x[:2], q, s, 40, ids)
    bad("x must be \\[tokens\\]", fq.fp4_gemv_mx, x[:, None], q, s, 40, ids)
    bad("first", fq.fp4_gemv_mx, x, q[0], s[0], 40, first=1)
    bad("first = -1", fq.fp4_gemv_mx, x, q, s, 40, ids, -1)
    bad("out must be", fq.fp4_gemv_mx, x, q[0], s[0], 40, out=torch.zeros((3, 40), device="cuda"))
    bad("equally far", fq.fp4_gemv_mx, x, q, s, 40, ids, out_dtype=torch.float32,
        out=torch.zeros((3, 3, 40), device="cuda")[:, :2])
    bad("overlap", fq.fp4_gemv_mx, x, q[0], s[0], 40, out_dtype=torch.float32, out=torch.zeros((1, 40), device="cuda").expand(3, 40))
    bad("unit stride", fq.fp4_gemv_mx, torch.zeros((3, 400), dtype=torch.bfloat16, device="cuda")[:, ::2], q[0], s[0], 40)
    bad("live on the GPU", fq.fp4_gemv_mx, x.cpu(), q[0], s[0], 40)
    bad("status 2", fq.fp4_gemv_mx, x[:1].repeat(200, 1), q, s, 40, ids[:1, :1].repeat(200, 33))
