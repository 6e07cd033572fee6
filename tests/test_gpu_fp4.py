"""GPU parity of the FP4 microscaling operators against the float64 oracle.

Quantization and read-back are exact: codes, scale bytes and values must equal
the oracle's. A product's error is bounded from its definition: the tile
products are added in FP32, so an output is off by at most one FP32 rounding of
the running sum (at most sum |a||b|) per tile of 128 and per joined partial,
doubled for the adds inside the matrix core; bf16 output adds half a unit in
its last place.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fine_grained_fp8_quantize_amd as fq
import workloads as wl
from gpu_util import dev_bf16, nan_out
from oracle import fp4

pytestmark = pytest.mark.gpu


def host_tiles(q, s):
    return q.cpu().numpy(), s.cpu().numpy().view(np.uint8).reshape(*s.shape, 4)


def dev_tiles(codes, ebytes):
    q, s = fp4.tiles(codes, ebytes)
    return torch.from_numpy(q).cuda(), torch.from_numpy(s.view(np.int32).reshape(s.shape[:3])).cuda()


def act(seed, rows, cols):
    return wl.activation(seed, "tiny_fprop", 120, rows, cols, 50.0)


def check_matrix(q, s, bits, what):
    ref_q, ref_s = fp4.tiles(*fp4.quantize(bits))
    got_q, got_s = host_tiles(q, s)
    assert np.array_equal(got_q, ref_q), what + " codes"
    assert np.array_equal(got_s, ref_s), what + " scale bytes"


SIZES = [(1, 1), (1, 32), (3, 31), (16, 128), (17, 129), (15, 512), (33, 520), (130, 1000), (64, 2048), (257, 96)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("tiling", ["1x32", "32x1"])
def test_quantize_and_read_back(rows, cols, tiling):
    bits = act(rows + cols, rows, cols)
    q, s = fq.fp4_quantize_mx(dev_bf16(bits), tiling)
    ref = bits if tiling == "1x32" else np.ascontiguousarray(bits.T)
    check_matrix(q, s, ref, tiling)
    want = fp4.values(*fp4.quantize(ref))[:, :ref.shape[1]]
    for dt in (torch.bfloat16, torch.float32):
        v = fq.fp4_dequantize_mx(q, s, *ref.shape, dt, out=nan_out(ref.shape, dt))
        assert np.array_equal(v.double().cpu().numpy(), want), dt


def test_quantize_special_blocks():
    rng = np.random.default_rng(3)
    rows = [np.zeros(160, np.uint16), np.full(160, 0x8000, np.uint16),            # zeros of both signs
            rng.integers(1, 0x80, 160).astype(np.uint16),                          # subnormals
            rng.integers(0x80, 0x200, 160).astype(np.uint16),                      # the clamp at 2^-127
            np.full(160, 0x7F7F, np.uint16),                                       # the largest values
            rng.integers(0, 0x7F80, 160).astype(np.uint16) | (rng.integers(0, 2, 160).astype(np.uint16) << 15)]
    for v in (0x7F80, 0xFF80, 0x7FC0, 0x7F81):                                     # infinities and NaNs
        r = wl.f32_to_bf16_bits(rng.standard_normal(160).astype(np.float32))
        r[70] = v
        rows.append(r)
    bits = np.stack(rows)
    for tiling, ref in (("1x32", bits), ("32x1", np.ascontiguousarray(bits.T))):
        x = dev_bf16(bits)
        q, s = fq.fp4_quantize_mx(x, tiling)
        check_matrix(q, s, ref, "special " + tiling)
        v = fq.fp4_dequantize_mx(q, s, *ref.shape, torch.float32).double().cpu().numpy()
        assert np.array_equal(v, fp4.values(*fp4.quantize(ref))[:, :ref.shape[1]], equal_nan=True)


def test_every_bf16_value_under_every_exponent_of_its_block():
    """All finite bf16 magnitudes beside block maxima of 24 exponents."""
    mags = np.arange(0x7F80, dtype=np.uint32)
    blocks = []
    for top in list(range(0, 16)) + [100, 127, 128, 200, 250, 252, 253, 254]:
        limit = (top << 7) | 0x7F
        v = mags[mags <= limit]
        v = v[:: max(1, len(v) // 4000)]
        v = np.concatenate([v, np.full(-len(v) % 31, 0)]).reshape(-1, 31)
        blocks.append(np.concatenate([v, np.full((len(v), 1), limit)], axis=1))
    bits = np.concatenate(blocks).astype(np.uint16)
    bits = np.concatenate([bits, bits[-(-len(bits) % 16) or len(bits):]]) if len(bits) % 16 else bits
    signs = np.random.default_rng(4).integers(0, 2, bits.shape).astype(np.uint16) << 15
    q, s = fq.fp4_quantize_mx(dev_bf16(bits | signs))
    check_matrix(q, s, bits | signs, "sweep")


@pytest.mark.parametrize("tiling", ["1x32", "32x1"])
def test_quantize_strided_and_unaligned_views(tiling):
    rows, cols = 50, 200
    bits = act(9, rows, cols)
    ref = bits if tiling == "1x32" else np.ascontiguousarray(bits.T)
    for ld, shift in ((208, 0), (201, 0), (208, 8), (208, 3), (333, 5)):
        buf = torch.zeros(rows * ld + shift + 16, dtype=torch.int16, device="cuda")
        view = buf[shift:shift + rows * ld].view(rows, ld)[:, :cols].view(torch.bfloat16)
        view.copy_(dev_bf16(bits))
        q, s = fq.fp4_quantize_mx(view, tiling)
        check_matrix(q, s, ref, "ld %d shift %d" % (ld, shift))


def test_quantize_into_a_range_of_row_tiles():
    bits = act(10, 20, 300)
    q = torch.full((3, 5, 1024), 7, dtype=torch.uint8, device="cuda")
    s = torch.full((1, 5, 64), 7, dtype=torch.int32, device="cuda")
    fq.fp4_quantize_mx(dev_bf16(bits), q=q[:, 1:3], scale=s[:, 1:3])
    check_matrix(q[:, 1:3], s[:, 1:3], bits, "window")
    assert (q[:, [0, 3, 4]] == 7).all() and (s[:, [0, 3, 4]] == 7).all(), "tiles outside the window written"
    v = fq.fp4_dequantize_mx(q[:, 1:3], s[:, 1:3], 20, 300, torch.float32).double().cpu().numpy()
    assert np.array_equal(v, fp4.values(*fp4.quantize(bits))[:, :300])


@pytest.mark.parametrize("tiling", ["1x32", "32x1"])
def test_quantize_a_stack(tiling):
    stack = np.stack([wl.weight(1, "tiny_fprop", 130 + e, 40, 600) for e in range(3)])
    x = dev_bf16(stack.reshape(120, 600)).view(3, 40, 600)
    q, s = fq.fp4_quantize_mx(x, tiling)
    for e in range(3):
        check_matrix(q[e], s[e], stack[e] if tiling == "1x32" else np.ascontiguousarray(stack[e].T), "matrix %d" % e)
    # a stack of strided views
    big = torch.zeros((3, 48, 608), dtype=torch.bfloat16, device="cuda")
    big[:, :40, :600] = x
    q2, s2 = fq.fp4_quantize_mx(big[:, :40, :600], tiling)
    assert torch.equal(q, q2) and torch.equal(s, s2)


def test_empty_sizes():
    for shape in ((0, 64), (64, 0)):
        x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        for tiling in ("1x32", "32x1"):
            q, s = fq.fp4_quantize_mx(x, tiling)
            assert q.numel() == 0 and s.numel() == 0
    q, s = fq.fp4_quantize_mx(torch.empty((5, 0), dtype=torch.bfloat16, device="cuda"))
    w, ws = fq.fp4_quantize_mx(torch.empty((7, 0), dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(fq.fp4_gemm_mx(q, s, w, ws, 5, 7, torch.float32, out=nan_out((5, 7), torch.float32)),
                       torch.zeros((5, 7), device="cuda"))
    q, s = fq.fp4_quantize_mx(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"))
    assert fq.fp4_gemm_mx(q, s, q, s).shape == (0, 0)
    assert fq.fp4_dequantize_mx(q, s, 0, 64).shape == (0, 64)


@pytest.mark.parametrize("tokens,cols,topk,m_total", [(1, 32, 1, 16), (19, 130, 3, 80), (100, 1030, 8, 900), (64, 512, 2, 128)])
def test_scatter(tokens, cols, topk, m_total):
    bits = act(11, tokens, cols)
    rng = np.random.default_rng(tokens)
    dst = np.full((tokens, topk), -1, np.int32)
    places = rng.permutation(m_total)[:tokens * topk // 2 + 1]
    dst.reshape(-1)[rng.permutation(tokens * topk)[:len(places)]] = places
    dst.reshape(-1)[rng.permutation(tokens * topk)[:1]] = m_total + 3          # past the layout: ignored
    codes, e = fp4.quantize(bits)
    ref_codes, ref_e = np.full((m_total, codes.shape[1]), 5, np.uint8), np.full((m_total, e.shape[1]), 9, np.uint8)
    q, s = dev_tiles(ref_codes, ref_e)
    fq.fp4_quantize_mx_scatter(dev_bf16(bits), torch.from_numpy(dst).cuda(), m_total, q=q, scale=s)
    for t in range(tokens):
        for r in dst[t]:
            if 0 <= r < m_total:
                ref_codes[r], ref_e[r] = codes[t], e[t]
    got = fq.fp4_dequantize_mx(q, s, m_total, cols, torch.float32).double().cpu().numpy()
    assert np.array_equal(got, fp4.values(ref_codes, ref_e)[:, :cols])


# ---------------------------------------------------------------- products

def bounds(a, b, out_dtype, joined=16):
    ref = a @ b.T
    mag = np.abs(a) @ np.abs(b).T
    e = (-(-a.shape[1] // 128) + joined) * 2.0 ** -23 * mag
    if out_dtype == torch.bfloat16:
        e = e + 2.0 ** -8 * (np.abs(ref) + e)  # 8 significant bits: half a unit is 2^-8 at most
    return ref, e + 1e-300


def gemm_case(m, n, k, out_dtype, seed=0):
    ab, bb = act(seed, m, k), wl.weight(seed, "tiny_fprop", 121, n, k)
    a, sa = fq.fp4_quantize_mx(dev_bf16(ab))
    b, sb = fq.fp4_quantize_mx(dev_bf16(bb))
    c = fq.fp4_gemm_mx(a, sa, b, sb, m, n, out_dtype, out=nan_out((m, n), out_dtype))
    ref, e = bounds(fp4.values(*fp4.quantize(ab)), fp4.values(*fp4.quantize(bb)), out_dtype)
    bad = np.abs(c.double().cpu().numpy() - ref) > e
    assert not bad.any(), "%d x %d x %d: %d outputs off, or not written" % (m, n, k, bad.sum())


SHAPES = [(1, 1, 1), (1, 16, 32), (1, 130, 4100), (2, 50, 128), (15, 64, 640), (16, 256, 512), (17, 33, 160),
          (31, 128, 1000), (33, 100, 2048), (63, 17, 96), (64, 512, 1024), (65, 300, 544), (100, 1, 513),
          (128, 128, 128), (129, 257, 384), (200, 700, 1536), (255, 256, 4096), (256, 256, 256), (257, 513, 1100),
          (300, 260, 65), (512, 768, 896), (520, 1030, 2176)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_gemm(m, n, k, out_dtype):
    gemm_case(m, n, k, out_dtype)


@pytest.mark.parametrize("m,n,k", [(1, 4096, 7168), (40, 2048, 8192), (1024, 1536, 7168), (2048, 7168, 1024)])
def test_gemm_large(m, n, k):
    gemm_case(m, n, k, torch.bfloat16, seed=1)


def test_gemm_transposed_operands_are_the_two_gradients():
    """dX = dY W and dW = dY^T X with the 32x1 operands."""
    tokens, n, k = 160, 96, 130
    dy, x, w = act(21, tokens, n), act(22, tokens, k), wl.weight(3, "tiny_fprop", 122, n, k)
    val = lambda bits: fp4.values(*fp4.quantize(np.ascontiguousarray(bits)))  # noqa: E731
    dx = fq.fp4_gemm_mx(*fq.fp4_quantize_mx(dev_bf16(dy)), *fq.fp4_quantize_mx(dev_bf16(w), "32x1"), tokens, k,
                        torch.float32)
    ref, e = bounds(val(dy), val(w.T), torch.float32)
    assert (np.abs(dx.double().cpu().numpy() - ref) <= e).all()
    dw = fq.fp4_gemm_mx(*fq.fp4_quantize_mx(dev_bf16(dy), "32x1"), *fq.fp4_quantize_mx(dev_bf16(x), "32x1"), n, k,
                        torch.float32)
    ref, e = bounds(val(dy.T), val(x.T), torch.float32)
    assert (np.abs(dw.double().cpu().numpy() - ref) <= e).all()


@pytest.mark.parametrize("m", [5, 70, 300])
def test_gemm_windows_and_strided_output(m):
    """Operands as ranges of row tiles of larger matrices, an output with any
    leading dimension and alignment; nothing outside it is written."""
    n, k = 50, 650
    ab, bb = act(31, m + 48, k), wl.weight(4, "tiny_fprop", 123, n + 64, k)
    a, sa = fq.fp4_quantize_mx(dev_bf16(ab))
    b, sb = fq.fp4_quantize_mx(dev_bf16(bb))
    rt = -(-m // 16)
    ref, e = bounds(fp4.values(*fp4.quantize(ab))[32:32 + m], fp4.values(*fp4.quantize(bb))[16:16 + n], torch.float32)
    for ld, shift in ((52, 0), (51, 0), (64, 4), (57, 3)):
        buf = torch.full((m * ld + shift + 8,), 3.0, device="cuda")
        out = buf[shift:shift + m * ld].view(m, ld)
        fq.fp4_gemm_mx(a[:, 2:2 + rt], sa[:, 2:2 + rt], b[:, 1:5], sb[:, 1:5], m, n, torch.float32, out=out[:, :n])
        assert (np.abs(out[:, :n].double().cpu().numpy() - ref) <= e).all(), (ld, shift)
        out[:, :n] = 3.0
        assert (buf == 3.0).all(), "written outside the output"


def test_gemm_nan_stays_in_its_rows():
    m, n, k = 40, 48, 300
    ab, bb = act(41, m, k), wl.weight(5, "tiny_fprop", 124, n, k)
    ab[7, 200] = 0x7FC0
    bb[33, 10] = 0x7F80
    c = fq.fp4_gemm_mx(*fq.fp4_quantize_mx(dev_bf16(ab)), *fq.fp4_quantize_mx(dev_bf16(bb)), m, n, torch.float32)
    want = np.zeros((m, n), bool)
    want[7], want[:, 33] = True, True
    assert np.array_equal(np.isnan(c.cpu().numpy()), want)


@pytest.mark.parametrize("m", [3, 129, 1024])
def test_gemm_repeats_bit_for_bit_and_on_another_stream(m):
    n, k = 1000, 4000
    a = fq.fp4_quantize_mx(dev_bf16(act(51, m, k)))
    b = fq.fp4_quantize_mx(dev_bf16(wl.weight(6, "tiny_fprop", 125, n, k)))
    first = fq.fp4_gemm_mx(*a, *b, m, n, torch.float32)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    again = [fq.fp4_gemm_mx(*a, *b, m, n, torch.float32, stream=side) for _ in range(3)]
    side.synchronize()
    assert all(torch.equal(first, c) for c in again)


# ----------------------------------------------------------------- experts

def grouped_case(rows, n, k, align, extra, out_dtype, with_rows=True, poison=True, seed=0):
    rows = np.asarray(rows, np.int64)
    off = wl.pad_offsets(rows, align)
    groups, m_total = len(rows), int(off[-1]) + extra
    ab = act(seed + 1, max(m_total, 1), k)[:m_total]
    wb = np.stack([wl.weight(seed, "tiny_fprop", 140 + e, n, k) for e in range(groups)])
    av = fp4.values(*fp4.quantize(ab))
    if poison:  # padding rows may hold anything
        for e in range(groups):
            ab[off[e] + rows[e]:off[e + 1], 0] = 0x7FC0
        ab[off[-1]:, 0] = 0x7FC0
    a, sa = fq.fp4_quantize_mx(dev_bf16(ab))
    b, sb = fq.fp4_quantize_mx(dev_bf16(wb.reshape(groups * n, k)).view(groups, n, k))
    c = fq.fp4_grouped_gemm_mx(torch.from_numpy(off.astype(np.int32)).cuda(),
                               torch.from_numpy(rows.astype(np.int32)).cuda() if with_rows else None, a, sa, b, sb, n,
                               out_dtype, out=nan_out((m_total, n), out_dtype)).double().cpu().numpy()
    real = np.zeros(m_total, bool)
    for e in range(groups):
        hi = off[e] + (rows[e] if with_rows else off[e + 1] - off[e])
        real[off[e]:hi] = True
        ref, tol = bounds(av[off[e]:hi], fp4.values(*fp4.quantize(wb[e])), out_dtype)
        assert (np.abs(c[off[e]:hi] - ref) <= tol).all(), "expert %d" % e
    assert (c[~real] == 0).all(), "padding rows not zero"


@pytest.mark.parametrize("rows,n,k,align,extra", [
    ([1], 16, 32, 16, 0), ([0, 0, 0], 33, 128, 16, 48), ([3, 0, 17, 1, 16, 0, 40], 100, 700, 16, 16),
    ([5, 130, 0, 64], 300, 1024, 128, 0), ([300, 5, 0, 128, 257, 40], 384, 640, 128, 256),
    ([1] * 70, 48, 256, 16, 0), ([0] * 66 + [33, 2], 64, 384, 16, 32), ([600, 0, 31], 530, 1300, 16, 400),
    ([256, 256], 256, 512, 128, 0), ([1000, 3], 256, 128, 16, 0)])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_grouped(rows, n, k, align, extra, out_dtype):
    grouped_case(rows, n, k, align, extra, out_dtype)


def test_grouped_without_row_counts():
    grouped_case([20, 0, 100, 7], 80, 300, 16, 32, torch.float32, with_rows=False, poison=False)


def test_grouped_keeps_to_its_rows_with_broken_offsets():
    """Offsets outside the contract give unspecified values inside C only."""
    a, sa = fq.fp4_quantize_mx(dev_bf16(act(61, 64, 256)))
    b, sb = fq.fp4_quantize_mx(dev_bf16(wl.weight(7, "tiny_fprop", 126, 64, 256)).view(2, 32, 256))
    buf = torch.full((64 + 32, 32), 3.0, device="cuda")
    for off in ([0, 4096, 64], [-160, 32, 1 << 30], [48, 16, 0], [7, 9, 33]):
        fq.fp4_grouped_gemm_mx(torch.tensor(off, dtype=torch.int32).cuda(), None, a, sa, b, sb, 32, torch.float32,
                               out=buf[16:80])
        assert (buf[:16] == 3).all() and (buf[80:] == 3).all(), off
