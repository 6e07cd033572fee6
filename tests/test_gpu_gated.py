"""The gated feed-forward operators on the GPU against the float64 oracle: few
rows and many, odd sizes and pitches, every output type, experts with and
without rows, padding, the gradients in both tilings."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fine_grained_fp8_quantize_amd as fq
from gpu_util import assert_bits_equal, assert_gemm_close, host_codes
from oracle import gated as model

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
U = 2.0 ** -24


def _bf16(rng, *shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16).cuda()


def _codes(rng, *shape):
    """Random E4M3 codes without a NaN, of values up to 240."""
    q = rng.integers(0, 0x78, shape) | (rng.integers(0, 2, shape) << 7)
    return q.astype(np.uint8)


def _problem(seed, m, n, k, lead=()):
    """Codes and scales whose products are of the order of one."""
    rng = np.random.default_rng(seed)
    a, b = _codes(rng, m, k), _codes(rng, *lead, 2, n, k)
    a_s = (rng.uniform(0.5, 2.0, (k // 128, m)) / 64).astype(np.float32)
    b_s = (rng.uniform(0.5, 2.0, (*lead, 2, -(-n // 128), k // 128)) / 64 / np.sqrt(k)).astype(np.float32)
    return a, a_s, b, b_s


def _dev(*xs):
    return [torch.from_numpy(x).cuda() for x in xs]


def _finite(t):
    return t.float().cpu().numpy().astype(np.float64)


def _close(got, ref, what):
    """The criteria of the framework's products. Their bar on the norm, 2e-3, stands for the mean of many roundings;
    one rounding to bf16 alone is up to 2^-8 of its value, and so is the norm of a few elements: 2^-8 + 2e-4, the
    second for the products' own sums (at most 7e-5 of values from the rms on in the accumulation study)."""
    if ref.size >= 4096:
        assert_gemm_close(got, ref, what)
        return
    rms = np.sqrt(np.mean(ref * ref)) if ref.size else 0.0
    assert np.all(np.isfinite(got)), what
    assert np.linalg.norm(got - ref) <= (2.0 ** -8 + 2e-4) * np.linalg.norm(ref), what
    assert np.all(np.abs(got - ref) <= 1e-2 * (np.abs(ref) + rms)), what


SHAPES = [(1, 128, 128), (1, 2048, 1024), (3, 8, 256), (16, 130, 384), (17, 129, 128), (33, 250, 640), (64, 100, 2048),
          (65, 128, 256), (130, 300, 384), (256, 128, 512), (300, 131, 128), (513, 384, 1152), (1, 1, 128), (2, 7, 7168), (90, 2100, 384), (2100, 521, 256), (4097, 260, 128)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_products(m, n, k, act):
    a, a_s, b, b_s = _problem(m * 7 + n, m, n, k)
    want, gate, up = model.block(act, a, a_s, b, b_s)
    d = _dev(a, a_s, b, b_s)
    for dt in (torch.bfloat16, torch.float32):
        keep = torch.full((m, 2 * n), float("nan"), dtype=torch.bfloat16, device="cuda")
        out = torch.full((m, n), float("nan"), dtype=dt, device="cuda")
        assert fq.fp8_gated_gemm(*d, act, dt, out=out, gate_up=keep) is out
        _close(_finite(out), want, "H")
        _close(_finite(keep[:, :n]), gate, "gate")
        _close(_finite(keep[:, n:]), up, "up")


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("m,n,k", [(1, 128, 256), (5, 256, 1024), (40, 384, 512), (70, 128, 384), (300, 256, 1280),
                                   (2300, 640, 256)])
def test_codes_are_those_of_the_fp32_result(m, n, k, act):
    d = _dev(*_problem(m + n, m, n, k))
    h = fq.fp8_gated_gemm(*d, act, torch.float32).cpu().numpy()
    want_q, want_s = model.tiles_1x128(h)
    q = torch.full((m, n + 16), 255, dtype=torch.uint8, device="cuda")
    s = torch.full((n // 128, m + 3), float("nan"), device="cuda")
    keep = torch.zeros((m, 2 * n), dtype=torch.bfloat16, device="cuda")
    fq.fp8_gated_gemm(*d, act, E4M3, out=q[:, :n], scale=s[:, :m], gate_up=keep)
    assert_bits_equal(host_codes(q)[:, :n], want_q, "codes")
    assert_bits_equal(s.cpu().numpy()[:, :m], want_s, "scales")
    assert (q[:, n:] == 255).all() and torch.isnan(s[:, m:]).all()
    # without scratch the tile kernel takes few rows too: its sums differ in order alone
    if m <= 64:
        q2, s2 = fq.fp8_gated_gemm(*d, act, E4M3, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
        v, v2 = model.values(host_codes(q)[:, :n], want_s, 1), model.values(host_codes(q2), s2.cpu().numpy(), 1)
        # one code apart at the most, where a sum lies next to the border of two
        step = np.maximum(np.abs(v) / 8, np.repeat(want_s.T, 128, 1) * 2.0 ** -9) * 1.001
        assert np.all(np.abs(v - v2) <= step) and np.mean(np.abs(v - v2) > 1e-3 * step) < 0.01


@pytest.mark.parametrize("m,n,k", [(2300, 640, 256), (4099, 384, 1152)])
def test_products_are_those_of_the_plain_gemm(m, n, k):
    """The same instructions in the same order: gate and up bit for bit, and H from them with the activation's few
    roundings (the logistic's power, its correction, sum and reciprocal, and two products: 8 last places)."""
    d = _dev(*_problem(3, m, n, k))
    keep = torch.empty((m, 2 * n), dtype=torch.bfloat16, device="cuda")
    h = _finite(fq.fp8_gated_gemm(*d, "silu", torch.float32, gate_up=keep))
    g, u = (fq.fp8_gemm(d[0], d[1], d[2][i].contiguous(), d[3][i].contiguous(), "block", torch.float32) for i in (0, 1))
    assert torch.equal(keep, torch.cat((g, u), 1).to(torch.bfloat16))
    want = model.act("silu", _finite(g)) * _finite(u)
    assert np.all(np.abs(h - want) <= 8 * 2 * U * np.abs(want) + 1e-30)


def test_extremes_of_the_activation():
    """Gates up to +-1e4: no overflow in the logistic, exact limits."""
    k, n = 128, 128
    a = np.full((64, k), 0x38, np.uint8)          # 1.0
    b = np.zeros((2, n, k), np.uint8)
    b[0, :, 0], b[1, :, 0] = 0x38, 0x38
    gates = np.concatenate([np.linspace(-100, 100, 62), [-1e4, 1e4]]).astype(np.float32)
    b_s = np.ones((2, 1, 1), np.float32)
    for act in ("silu", "gelu"):
        h = _finite(fq.fp8_gated_gemm(*_dev(a, gates.reshape(1, 64), b, b_s), act, torch.float32))[:, 0]
        x = gates.astype(np.float64)
        with np.errstate(over="ignore"):
            want = model.act(act, x) * x
        # gelu's argument: three products and a sum before the logistic, |w| 4 U relative to what it decides
        w = np.abs(x) if act == "silu" else 1.6 * (np.abs(x) + 0.045 * np.abs(x) ** 3)
        assert np.all(np.abs(h - want) <= (16 + 4 * (act == "gelu") * np.minimum(w, 88)) * U * np.abs(want) + 1e-30), act


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gates_of_any_size(act):
    """Gates whose powers pass FP32: the activation is g or 0 there, its slope 1 or 0."""
    k, n = 128, 128
    big = np.array([17.0, 90.0, 300.0, 5e12, 1e13, 3e19, 1e25, 1e38], np.float32)
    gates = np.concatenate([big, -big])
    a = np.full((16, k), 0x38, np.uint8)          # 1.0
    b = np.zeros((2, n, k), np.uint8)
    b[0, :, 0], b[1, :, 0] = 0x38, 0x38
    b_s = np.array([1.0, 2e-38], np.float32).reshape(2, 1, 1)
    d = _dev(np.repeat(a, 5, 0), np.tile(gates, 5).reshape(1, 80), b, b_s)
    x = gates.astype(np.float64)
    with np.errstate(over="ignore"):
        want = model.act(act, x) * x * float(b_s[1, 0, 0])
    # (act(-17) is the smallest that is not 0 for both: 7e-7 of it; gelu's argument as in the test above)
    room = (16 + 4 * 88) * U * np.abs(want) + 1e-38
    for m in (16, 80):
        h = _finite(fq.fp8_gated_gemm(d[0][:m], d[1][:, :m], *d[2:], act, torch.float32))
        assert np.all(np.abs(h - np.tile(want, m // 16)[:, None]) <= np.tile(room, m // 16)[:, None]), m
    for m, cols in ((16, 128), (128, 128)):
        g = torch.from_numpy(gates).to(torch.bfloat16).cuda().repeat(m // 16)[:, None].expand(m, cols)
        one = torch.full((m, cols), 0.5, dtype=torch.bfloat16, device="cuda")
        got = _finite(fq.fp8_gated_backward(one, torch.cat((g, one), 1), act, torch.bfloat16))
        y = _finite(g)[:16, :1]
        with np.errstate(over="ignore"):
            dg, du = model.gradients(act, np.full_like(y, 0.5), y, np.full_like(y, 0.5))
        want2 = np.tile(np.concatenate((np.repeat(dg, cols, 1), np.repeat(du, cols, 1)), 1), (m // 16, 1))
        # bf16's rounding, and the slope's terms past -17 of either sign: 17 * 4e-8 and less
        assert np.all(np.abs(got - want2) <= 2.0 ** -8 * 1.001 * np.abs(want2) + 16 * U * 17), m
        outs = fq.fp8_gated_backward(one, torch.cat((g, one), 1), act, transposed=m == 128)
        for t in outs[1::2]:
            assert torch.isfinite(t).all()
        for t in outs[0::2]:
            assert ((t.view(torch.uint8) & 127) != 127).all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_a_nan_stays_in_its_element(act):
    rng = np.random.default_rng(8)
    dh, gu = _bf16(rng, 40, 100), _bf16(rng, 40, 200)
    clean = fq.fp8_gated_backward(dh, gu, act, torch.bfloat16)
    gu[3, 7], gu[5, 109], dh[6, 11] = float("nan"), float("nan"), float("nan")
    got = fq.fp8_gated_backward(dh, gu, act, torch.bfloat16)
    bad = torch.zeros_like(got, dtype=torch.bool)
    for row, col in ((3, 7), (3, 107), (5, 9), (6, 11), (6, 111)):
        bad[row, col] = True
    assert torch.equal(torch.isnan(got), bad) and torch.equal(got[~bad], clean[~bad])
    d = _dev(*_problem(8, 20, 100, 128))
    clean = fq.fp8_gated_gemm(*d, act)
    d[0][4, 5] = 0x7F
    got = fq.fp8_gated_gemm(*d, act)
    assert torch.isnan(got[4]).all() and torch.equal(got[:4], clean[:4]) and torch.equal(got[5:], clean[5:])


def test_strides_and_padded_operands():
    m, n, k = 100, 200, 256
    a, a_s, b, b_s = _problem(9, m, n, k)
    want, gate, up = model.block("silu", a, a_s, b, b_s)
    da = torch.zeros((m, k + 32), dtype=torch.uint8, device="cuda")
    da[:, :k] = torch.from_numpy(a)
    das = torch.full((k // 128, m + 5), float("nan"), device="cuda")
    das[:, :m] = torch.from_numpy(a_s)
    db = torch.zeros((2, n + 3, k + 16), dtype=torch.uint8, device="cuda")
    db[:, :n, :k] = torch.from_numpy(b)
    dbs = torch.full((2, 5, k // 128 + 1), float("nan"), device="cuda")
    dbs[:, :2, :k // 128] = torch.from_numpy(b_s)
    keep = torch.full((m, 2 * n + 16), float("nan"), dtype=torch.bfloat16, device="cuda")
    out = torch.full((m, n + 24), float("nan"), device="cuda")
    for rows in (m, 20):
        fq.fp8_gated_gemm(da[:rows, :k], das[:, :rows], db[:, :n, :k], dbs[:, :2, :k // 128], "silu", torch.float32,
                          out=out[:rows, :n], gate_up=keep[:rows, :2 * n])
        _close(_finite(out[:rows, :n]), want[:rows], "H")
        _close(_finite(keep[:rows, :n]), gate[:rows], "gate")
        assert torch.isnan(out[:, n:]).all() and torch.isnan(keep[:, 2 * n:]).all()
        out.fill_(float("nan"))
        keep.fill_(float("nan"))
    # the up weights in front of the gate's: any layout of two matrices
    both = torch.from_numpy(b[::-1].copy()).cuda()
    flipped = torch.as_strided(both, (2, n, k), (0, k, 1))
    got = fq.fp8_gated_gemm(*_dev(a, a_s), flipped, torch.from_numpy(b_s).cuda())
    want = model.block("silu", a, a_s, np.stack([b[1], b[1]]), b_s)[0]
    _close(_finite(got), want, "one matrix as both")


def test_empty_sizes():
    for m, n, k in ((0, 128, 128), (5, 0, 128), (5, 128, 0), (300, 128, 0)):
        a, a_s, b, b_s = _problem(1, m, n, max(k, 128))
        d = _dev(a[:, :k].copy(), a_s[:k // 128].copy(), b[..., :k].copy(), b_s[..., :k // 128].copy())
        keep = torch.full((m, 2 * n), float("nan"), dtype=torch.bfloat16, device="cuda")
        got = fq.fp8_gated_gemm(*d, gate_up=keep)
        assert got.shape == (m, n) and (got == 0).all() and (keep == 0).all()
        if n % 128 == 0:
            q, s = fq.fp8_gated_gemm(*d, out_dtype=E4M3)
            assert (q.view(torch.uint8) & 127 == 0).all() and (s == 0).all()


EXPERTS = [([130, 0, 1, 128], 0), ([256, 300, 64, 5, 0, 0], 128), ([0, 0], 256), ([700], 0), ([1] * 70, 0), ([385, 520, 1000, 257], 0),
           ([300, 641, 300], 384)]


COLUMNS = [(128, 256), (256, 1152), (200, 384), (7, 128), (2176, 256), (2300, 128)]


@pytest.mark.parametrize("rows,more", EXPERTS)
@pytest.mark.parametrize("n,k", COLUMNS)
def test_experts(rows, more, n, k):
    """`more`: rows set aside behind the last expert's, which are its padding."""
    rows = np.array(rows)
    off = np.concatenate([[0], np.cumsum(-(-rows // 128) * 128)])
    off[-1] += more
    m = int(off[-1])
    a, a_s, b, b_s = _problem(len(rows) + n, m, n, k, (len(rows),))
    real = np.zeros(m, bool)
    want, gate, up = (np.zeros((m, n)) for _ in range(3))
    for e in range(len(rows)):
        at = slice(off[e], off[e] + rows[e])
        real[at] = True
        want[at], gate[at], up[at] = model.block("silu", a[at], a_s[:, at], b[e], b_s[e])
    a[~real] = 0x7F  # NaN codes in the padding
    a_s[:, ~real] = np.nan
    d = _dev(off.astype(np.int32), rows.astype(np.int32), a, a_s, b, b_s)
    for dt in (torch.bfloat16, torch.float32):
        keep = torch.full((m, 2 * n), float("nan"), dtype=torch.bfloat16, device="cuda")
        out = torch.full((m, n), float("nan"), dtype=dt, device="cuda")
        fq.fp8_grouped_gated_gemm(*d, "silu", dt, out=out, gate_up=keep)
        for got, ref, what in ((out, want, "H"), (keep[:, :n], gate, "gate"), (keep[:, n:], up, "up")):
            got = _finite(got)
            assert np.all(got[~real] == 0) and np.all(np.isfinite(got)), what
            if real.any():
                _close(got[real], ref[real], what)
    if n % 128 == 0:
        h = _finite(out).astype(np.float32)
        want_q, want_s = model.tiles_1x128(h)
        q, s = fq.fp8_grouped_gated_gemm(*d, "silu", E4M3)
        assert_bits_equal(host_codes(q)[real], want_q[real], "codes")
        assert_bits_equal(s.cpu().numpy(), want_s, "scales")
        assert np.all(host_codes(q)[~real] & 127 == 0)
        # without scratch the tile kernel takes few rows too (see above: one code apart at the most)
        none = torch.empty(0, dtype=torch.uint8, device="cuda")
        q2, s2 = fq.fp8_grouped_gated_gemm(*d, "silu", E4M3, workspace=none)
        v, v2 = model.values(host_codes(q), want_s, 1), model.values(host_codes(q2), s2.cpu().numpy(), 1)
        step = np.maximum(np.abs(v) / 8, np.repeat(want_s.T, 128, 1) * 2.0 ** -9) * 1.001
        assert np.all(np.abs(v - v2) <= step) and np.mean(np.abs(v - v2) > 1e-3 * step) < 0.01
        assert np.all(host_codes(q2)[~real] & 127 == 0) and np.all(s2.cpu().numpy()[:, ~real] == 0)
    if (rows == np.diff(off)).all():
        assert torch.equal(fq.fp8_grouped_gated_gemm(d[0], None, *d[2:], "silu", dt), out)


def _room(act, dh, g, u):
    """What float32 leaves of the gradients: the logistic of w has its power's, its correction's, its sum's and its
    reciprocal's last places, and w's own (none for silu, 4 for gelu) times |w| (1 - s); 1 - s, the product with g
    and the slope's sum make 16 on |g| s + s at the most."""
    w = np.abs(g) if act == "silu" else 1.6 * (np.abs(g) + 0.045 * np.abs(g) ** 3)
    more = 0 if act == "silu" else 4 * np.minimum(w, 88)
    wide = 1.0 if act == "silu" else 1.6 * (1 + 0.135 * g * g)
    s = 1 / (1 + np.exp(-np.clip(g if act == "silu" else 1.596 * (g + 0.044715 * g ** 3), -80, 80)))
    return ((24 + 2 * more) * U * np.abs(dh * u) * s * (1 + np.abs(g) * wide) + 1e-37,
            (16 + more) * U * np.abs(dh * g) * s + 1e-37)


def _half_steps(v, scale):
    """Half a step of E4M3 at each value: 2^-4 of it, at least 2^-10 of the scale."""
    return np.maximum(np.abs(v) * 2.0 ** -4, scale * 2.0 ** -10)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("m,n,transposed", [(1, 128, False), (37, 256, False), (203, 512, False), (128, 128, True),
                                            (256, 384, True), (640, 128, True)])
def test_gradients_in_codes(m, n, transposed, act):
    rng = np.random.default_rng(m + n)
    dh, gu = _bf16(rng, m, n + 8, scale=1e-3)[:, :n], _bf16(rng, m, 2 * n + 24, scale=3.0)[:, :2 * n]
    x = [_finite(t) for t in (dh, gu[:, :n], gu[:, n:])]
    want = np.concatenate(model.gradients(act, *x), 1)
    room = np.concatenate(_room(act, *x), 1)
    out = fq.fp8_gated_backward(dh, gu, act, transposed=transposed)
    pairs = [(out[0], out[1], want, room)]
    if transposed:
        pairs.append((out[2], out[3], want.T, room.T))
    for q, s, ref, err in pairs:
        s = s.cpu().numpy().astype(np.float64)
        top = np.abs(ref).reshape(ref.shape[0], -1, 128)
        at = top.argmax(2)
        most = np.take_along_axis(top, at[..., None], 2)[..., 0]
        most_err = err.reshape(top.shape).max(2)
        assert np.all(np.abs(s.T * 448 - most) <= most_err + 2 * U * most)
        full = np.repeat(s.T, 128, 1)
        v = model.values(host_codes(q), s.astype(np.float32), 1)
        assert np.all(np.abs(v - ref) <= _half_steps(ref, full) * 1.0001 + 1.1 * err + 4 * U * np.abs(ref))
    # the same FP32 values in both: the plain call and the one with both tilings agree bit for bit along the rows
    if transposed:
        q, s = fq.fp8_gated_backward(dh, gu, act)
        assert_bits_equal(host_codes(q), host_codes(out[0]), "codes")
        assert_bits_equal(s.cpu().numpy(), out[1].cpu().numpy(), "scales")


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("m,n", [(1, 1), (3, 7), (37, 130), (64, 256), (129, 1000)])
@pytest.mark.parametrize("shift", [0, 1])
def test_gradients_in_bf16(m, n, act, shift):
    rng = np.random.default_rng(m * 31 + n)
    dh, gu = _bf16(rng, m, n + shift, scale=1e-3)[:, shift:], _bf16(rng, m, 2 * n + shift, scale=3.0)[:, shift:]
    x = [_finite(t) for t in (dh, gu[:, :n], gu[:, n:])]
    want, room = np.concatenate(model.gradients(act, *x), 1), np.concatenate(_room(act, *x), 1)
    got = _finite(fq.fp8_gated_backward(dh, gu, act, torch.bfloat16))
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * 1.001 * np.abs(want) + 1.01 * room)


def test_forward_and_gradient_agree_with_differences():
    """A step h along a random direction of gate and up changes sum(dH * H) by the gradients' product with it, but
    for h^2 times the third derivative: central differences in float64 of the oracle, the operator's gradient."""
    rng = np.random.default_rng(5)
    for act in ("silu", "gelu"):
        dh, gu = _bf16(rng, 64, 128), _bf16(rng, 64, 256, scale=2.0)
        d = _finite(fq.fp8_gated_backward(dh, gu, act, torch.bfloat16))
        x, y, dirn = _finite(dh), _finite(gu), rng.standard_normal((64, 256))
        f = lambda t: np.sum(x * model.act(act, (y + t * dirn)[:, :128]) * (y + t * dirn)[:, 128:])  # noqa: E731
        diff = (f(1e-4) - f(-1e-4)) / 2e-4
        assert abs(diff - np.sum(d * dirn)) <= 2.0 ** -8 * np.sqrt(np.sum((d * dirn) ** 2)) * 6 + 1e-4


def test_a_training_step_of_the_block():
    """Forward and backward of the whole block as a program runs it, against float64 on the operands' values."""
    m, n, k = 256, 128, 256
    rng = np.random.default_rng(11)
    x, dy = _bf16(rng, m, k), _bf16(rng, m, k, scale=1e-2)
    w, down = _bf16(rng, 2 * n, k, scale=0.06), _bf16(rng, k, n, scale=0.09)
    xq, xs = fq.fp8_quantize_act(x)
    wq, ws, wt, wts = fq.fp8_quantize_weight(w, transposed=True)
    dq, ds, dt, dts = fq.fp8_quantize_weight(down, transposed=True)
    keep = torch.empty((m, 2 * n), dtype=torch.bfloat16, device="cuda")
    h, hs = fq.fp8_gated_gemm(xq, xs, wq.view(2, n, k), ws.view(2, n // 128, k // 128), "silu", E4M3, gate_up=keep)
    y = fq.fp8_gemm(h, hs, dq, ds, "block", torch.float32)
    dyq, dys = fq.fp8_quantize_act(dy)
    dh = fq.fp8_gemm(dyq, dys, dt, dts, "block", torch.bfloat16)
    g, gs, gt, gts = fq.fp8_gated_backward(dh, keep, transposed=True)
    dx = fq.fp8_gemm(g, gs, wt, wts, "block", torch.float32)
    xt, xts = fq.fp8_quantize_act(x, "128x1")
    dw = fq.fp8_gemm(gt, gts, xt, xts, "row", torch.float32)
    # float64, from the same codes of x, W and dY on; what is rounded in between: H and the gradients to E4M3 (2^-4),
    # gate, up and dH to bf16
    xv, wv = model.values(host_codes(xq), xs.cpu().numpy(), 1), model.values(host_codes(wq), ws.cpu().numpy(), 128)
    dv, dyv = model.values(host_codes(dq), ds.cpu().numpy(), 128), model.values(host_codes(dyq), dys.cpu().numpy(), 1)
    gate, up = xv @ wv[:n].T, xv @ wv[n:].T
    hv = model.act("silu", gate) * up
    dg, du = model.gradients("silu", dyv @ dv, gate, up)
    d = np.concatenate((dg, du), 1)
    xtv = model.values(host_codes(xt), xts.cpu().numpy(), 1).T
    for got, ref, what in ((y, hv @ dv.T, "y"), (dx, d @ wv, "dx"), (dw, d.T @ xtv, "dw")):
        got = _finite(got)
        # rounding errors of E4M3 are independent, each at most 2^-4 of its term: 2^-4 normwise bounds their sum
        assert np.linalg.norm(got - ref) <= 2.0 ** -4 * np.linalg.norm(ref), what


def test_streams_and_replays():
    m, n, k = 128, 256, 512
    d = [_dev(*_problem(s, m, n, k)) for s in (1, 2)]
    rng = np.random.default_rng(3)
    dh = [_bf16(rng, m, n) for _ in range(2)]

    def step(i, bufs):
        q, s, keep = bufs[:3]
        fq.fp8_gated_gemm(*d[i], "gelu", E4M3, out=q, scale=s, gate_up=keep)
        fq.fp8_gated_gemm(d[i][0][:9], d[i][1][:, :9], *d[i][2:], "gelu", out=bufs[3])
        fq.fp8_gated_backward(dh[i], keep, "gelu", transposed=True, out=bufs[4], scale=bufs[5], out_t=bufs[6],
                              scale_t=bufs[7])

    def buffers():
        f = lambda *s, dt=torch.uint8: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
        return [f(m, n), f(n // 128, m, dt=torch.float32), f(m, 2 * n, dt=torch.bfloat16), f(9, n, dt=torch.bfloat16),
                f(m, 2 * n), f(n // 64, m, dt=torch.float32), f(2 * n, m), f(m // 128, 2 * n, dt=torch.float32)]

    want = [buffers(), buffers()]
    for i in (0, 1):
        step(i, want[i])
    torch.cuda.synchronize()
    got, streams = [buffers(), buffers()], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                step(i, got[i])
    torch.cuda.synchronize()
    graph, replayed = torch.cuda.CUDAGraph(), buffers()
    with torch.cuda.graph(graph):
        step(0, replayed)
    for _ in range(3):
        for b in replayed:
            b.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(replayed, want[0]):
            assert torch.equal(x, y)
    for i in (0, 1):
        for x, y in zip(got[i], want[i]):
            assert torch.equal(x, y)


def test_a_stream_of_its_own_and_experts_in_a_graph():
    """`stream=`: outputs and scratch of two calls at once; experts' few rows captured, with scratch of the graph."""
    rows = np.array([3, 0, 128, 40])
    off = np.concatenate([[0], np.cumsum(-(-rows // 128) * 128)])
    n, k = 256, 512
    d = [_dev(off.astype(np.int32), rows.astype(np.int32), *_problem(s, int(off[-1]), n, k, (4,))) for s in (1, 2)]
    few = [_dev(*_problem(s, 9, n, k)) for s in (3, 4)]
    run = lambda i, **kw: (*fq.fp8_grouped_gated_gemm(*d[i], "gelu", E4M3, **kw),  # noqa: E731
                           *fq.fp8_gated_gemm(*few[i], "silu", E4M3, **kw), fq.fp8_grouped_gated_gemm(*d[i], **kw))
    want = [[t.clone() for t in run(i)] for i in (0, 1)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[run(i, stream=streams[i]) for i in (0, 1)] for _ in range(4)]
    torch.cuda.synchronize()
    same = lambda x, y: torch.equal(x.view(torch.uint8), y.view(torch.uint8))  # noqa: E731
    for pair in got:
        for i in (0, 1):
            assert all(same(x, y) for x, y in zip(pair[i], want[i]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = run(0)
    for _ in range(3):
        for t in kept:
            t.view(torch.uint8).zero_()
        graph.replay()
        run(1)
        torch.cuda.synchronize()
        assert all(same(x, y) for x, y in zip(kept, want[0]))


def test_refusals():
    d = _dev(*_problem(1, 16, 200, 256))
    E = fq.Fp8qError
    bad = lambda match, *args, **kw: pytest.raises(E, fq.fp8_gated_gemm, *args, **kw).match(match)  # noqa: E731
    bad("act", *d, "relu")
    bad("out_dtype", *d, "silu", torch.float16)
    bad("whole 1x128 tiles", *d, "silu", E4M3)
    bad("scale belongs", *d, scale=d[1])
    bad("E4M3 codes", d[0].float(), *d[1:])
    bad("gate first", d[0], d[1], d[2][0], d[3][0])
    bad("disagree on K", d[0][:, :128], d[1][:1], *d[2:])
    bad("b_scale has shape", d[0], d[1], d[2], d[3][:, :1])
    bad("a_scale has shape", d[0], d[1][:, :8], *d[2:])
    bad("gate_up has", *d, gate_up=torch.zeros((16, 200), dtype=torch.bfloat16, device="cuda"))
    bad("out has dtype", *d, out=torch.zeros((16, 200), device="cuda"))
    bad("workspace", *d, workspace=torch.zeros(16, device="cuda"))
    bad("live on the GPU", d[0].cpu(), *d[1:])
    with pytest.raises(E, match="status 3"):
        fq.fp8_gated_gemm(*_dev(*_problem(1, 16, 128, 256)), out_dtype=E4M3,
                          out=torch.zeros((16, 136), dtype=torch.uint8, device="cuda")[:, 8:])
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(E, match="group_offsets"):
        fq.fp8_grouped_gated_gemm(off[:1], None, d[0], d[1], d[2][None], d[3][None])
    with pytest.raises(E, match="status 2"):
        fq.fp8_grouped_gated_gemm(off, None, d[0], d[1], d[2][None], d[3][None])
    x, gu = torch.zeros((20, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros((20, 256), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(E, match="whole 128x1 tiles"):
        fq.fp8_gated_backward(x, gu, transposed=True)
    with pytest.raises(E, match="gate_up has shape"):
        fq.fp8_gated_backward(x, gu[:, :128])
    with pytest.raises(E, match="belong to E4M3"):
        fq.fp8_gated_backward(x, gu, out_dtype=torch.bfloat16, transposed=True)
    with pytest.raises(E, match="whole 1x128"):
        fq.fp8_gated_backward(x[:, :100], gu[:, :200].contiguous())
    with pytest.raises(E, match="dh must be bfloat16"):
        fq.fp8_gated_backward(x.float(), gu)


def test_debug_checks_of_the_segments(monkeypatch):
    """FP8Q_DEBUG=1: segment arrays that break the contract are refused before the launch."""
    m, n, k = 256, 128, 128
    a, a_s, b, b_s = _problem(1, m, n, k, (2,))
    d = _dev(a, a_s, b, b_s)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    monkeypatch.setenv("FP8Q_DEBUG", "1")
    fq.fp8_grouped_gated_gemm(i32(0, 128, 256), i32(5, 128), *d)
    for off, rows in (((0, 64, 256), (5, 5)), ((0, 256, 128), (5, 5)), ((0, 128, 128), (5, 0)), ((128, 128, 256), (0, 5)),
                      ((0, 128, 256), (129, 5)), ((0, 128, 256), (-1, 5))):
        with pytest.raises(fq.Fp8qError, match="status 2"):
            fq.fp8_grouped_gated_gemm(i32(*off), i32(*rows), *d)
