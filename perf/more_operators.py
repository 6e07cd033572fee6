"""Workloads of the gated feed-forward block, from its training step to its serving: the FP8 gated products with
their gradient, the weight-only FP4 products of few tokens, and the optimizer step of the weights.

``listed()`` names the cases, ``draw()`` makes more of the same ranges, ``prepare()`` builds a case's inputs on the
GPU, ``run()`` makes one pass: in plain torch operations where ``own`` is false, through the package where it is true.
``exact()`` gives the same outputs in 64 bits.

* ``gated``: h = act(A Wg^T) (A Wu^T). A is E4M3 ``[m][k]`` with FP32 scales ``[k/128][m]`` (1x128 tiles); the weights
  are E4M3 ``[2][n][k]``, gate first, with scales ``[2][ceil(n/128)][ceil(k/128)]`` (128x128 blocks).
  ``keep``: gate and up in bf16 ``[m][2n]`` too, as the backward pass takes them.
* ``ffn``: the same with h quantized to E4M3 in 1x128 tiles, and the down product of that.
* ``experts``: the gated products of experts over rows sorted by expert, segments of whole 128 rows.
* ``backward``: the gradients of gate and up, quantized in 1x128 tiles and, with ``transposed``, in 128x1 tiles too.
* ``gemv``: bf16 rows times FP4 weights, plain or gated, of one matrix or of the experts that ``ids`` name. FP4 matrices
  are held in tiles of 16 rows x 128 k (1 KB): ``q`` is uint8 ``[kt][rt][1024]``, row r of a tile at byte 64 r and its
  32-element block b (16 bytes, low nibble first) at 16 * (b ^ ((r >> 2) & 3)) inside the row; ``scale`` is int32
  ``[ceil(kt/4)][rt][64]``, word 4 r + b holding the E8M0 bytes of block b of four consecutive k tiles.
* ``adamw``: one step over many tensors, FP32 parameters with a bf16 copy, bf16 gradients, states in 32 bits or in 8
  (the first moment and the root of the second as E4M3 codes with an FP32 scale for each 128 elements, rounded
  stochastically by a hash of seed, step, tensor and element).
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

_MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one token through a dense block's first half in FP8
        {"name": "gated_1x2048x7168", "op": "gated", "m": 1, "n": 2048, "k": 7168, "act": "silu", "keep": False},
        # a small training batch of odd sizes
        {"name": "gated_37x1000x1024", "op": "gated", "m": 37, "n": 1000, "k": 1024, "act": "gelu", "keep": True},
        # the forward pass of a dense block in training
        {"name": "ffn_4096x2048x7168", "op": "ffn", "m": 4096, "n": 2048, "k": 7168, "act": "silu"},
        # the local experts of a training step: 8192 routed rows, experts of uneven popularity
        {"name": "experts_8192x2048x7168", "op": "experts", "rows": 8192, "experts": 32, "skew": 0.6, "n": 2048,
         "k": 7168, "act": "silu"},
        # the gradient of a small batch of an odd number of tokens
        {"name": "backward_203x512", "op": "backward", "m": 203, "n": 512, "act": "gelu", "transposed": False},
        # the gradient of a training step, for both products that follow
        {"name": "backward_8192x2048", "op": "backward", "m": 8192, "n": 2048, "act": "silu", "transposed": True},
        # serving: one token through the down projection
        {"name": "gemv_1x7168x2048", "op": "gemv", "m": 1, "n": 7168, "k": 2048, "gated": False, "out": "bf16"},
        # serving: a few tokens through gate and up, odd sizes, fp32 output
        {"name": "gemv_gated_5x2050x7136", "op": "gemv", "m": 5, "n": 2050, "k": 7136, "gated": True, "act": "silu",
         "out": "f32"},
        # serving: 16 tokens through the gate and up of 4 of 32 experts each
        {"name": "gemv_experts_16x2048x7168", "op": "gemv", "m": 16, "n": 2048, "k": 7168, "gated": True,
         "act": "silu", "out": "bf16", "experts": 32, "topk": 4},
        # the many small tensors of a model: norms, biases, routers
        {"name": "adamw_small", "op": "adamw", "tensors": 120, "numel": 2000000, "bits": 32, "step": 3},
        # a layer's weights, states in 32 bits
        {"name": "adamw_64m", "op": "adamw", "tensors": 9, "numel": 64000000, "bits": 32, "step": 1000},
        # an expert layer's weights, states in 8 bits
        {"name": "adamw_8bit_128m", "op": "adamw", "tensors": 31, "numel": 128000000, "bits": 8, "step": 1000},
    ]


def _log_int(rng: random.Random, lo: int, hi: int) -> int:
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng: random.Random):
    op = rng.choice(["gated", "ffn", "experts", "backward", "gemv", "gemv", "adamw", "adamw"])
    act = rng.choice(["silu", "gelu"])
    if op == "gated":
        return {"op": op, "m": _log_int(rng, 1, 4096), "n": _log_int(rng, 16, 2048), "k": 128 * _log_int(rng, 1, 56),
                "act": act, "keep": rng.choice([False, True])}
    if op == "ffn":
        return {"op": op, "m": _log_int(rng, 1, 4096), "n": 128 * _log_int(rng, 1, 16), "k": 128 * _log_int(rng, 1, 56),
                "act": act}
    if op == "experts":
        experts = rng.choice([4, 8, 31, 32])
        return {"op": op, "rows": _log_int(rng, 1, 8192), "experts": experts, "skew": rng.choice([0.0, 0.6, 1.1]),
                "n": _log_int(rng, 64, 2048), "k": 128 * _log_int(rng, 1, 56), "act": act}
    if op == "backward":
        transposed = rng.choice([False, True])
        return {"op": op, "m": 128 * _log_int(rng, 1, 64) if transposed else _log_int(rng, 1, 8192),
                "n": 128 * _log_int(rng, 1, 16), "act": act, "transposed": transposed}
    if op == "gemv":
        case = {"op": op, "m": _log_int(rng, 1, 16), "n": _log_int(rng, 16, 7168), "k": _log_int(rng, 32, 7168),
                "gated": rng.choice([False, True]), "act": act, "out": rng.choice(["bf16", "f32"])}
        if rng.random() < 0.4:
            case["n"] = _log_int(rng, 16, 2048)
            case["experts"] = rng.choice([4, 8, 31, 32])
            case["topk"] = rng.randint(1, 4)
        return case
    return {"op": op, "tensors": _log_int(rng, 1, 120), "numel": _log_int(rng, 1000, 64000000),
            "bits": rng.choice([8, 32]), "step": _log_int(rng, 1, 100000)}


# ----------------------------------------------------------------- helpers

def _up(v: int, to: int) -> int:
    return -(-v // to) * to


def _dtype(name: str):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _gen(seed: int) -> torch.Generator:
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activation(g, rows: int, cols: int) -> torch.Tensor:
    """N(0, 1) with one entry in a thousand ten times larger."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    big = torch.rand((rows, cols), generator=g, device="cuda") < 1e-3
    return torch.where(big, x * 10.0, x)


def _plain_quantize_rows(x: torch.Tensor):
    """fp32 [rows][cols], cols % 128 == 0 -> E4M3 codes and scales [cols/128][rows] (1x128 tiles)."""
    b = x.reshape(x.shape[0], -1, 128)
    s = b.abs().amax(dim=2) / 448.0
    y = b / torch.where(s > 0, s, torch.ones_like(s)).unsqueeze(2)
    return y.reshape(x.shape).to(_E4M3), s.t().contiguous()


def _plain_rows(q: torch.Tensor, scale: torch.Tensor) -> torch.Tensor:
    """The fp32 values of codes [rows][cols] with scales [cols/128][rows]."""
    b = q.float().reshape(q.shape[0], -1, 128)
    return (b * scale.t().unsqueeze(2)).reshape(q.shape)


def _quantize_blocks(w: torch.Tensor):
    """[..][n][k] -> E4M3 codes and scales [..][ceil(n/128)][ceil(k/128)] (128x128 blocks)."""
    n, k = w.shape[-2:]
    p = torch.nn.functional.pad(w, (0, _up(k, 128) - k, 0, _up(n, 128) - n))
    b = p.reshape(*w.shape[:-2], _up(n, 128) // 128, 128, _up(k, 128) // 128, 128)
    s = b.abs().amax(dim=(-3, -1)) / 448.0
    q = (b / s.unsqueeze(-1).unsqueeze(-3)).reshape(p.shape)[..., :n, :k]
    return q.to(_E4M3).contiguous(), s.contiguous()


def _plain_blocks(q: torch.Tensor, scale: torch.Tensor) -> torch.Tensor:
    """The fp32 values of codes [..][n][k] with block scales."""
    n, k = q.shape[-2:]
    s = scale.repeat_interleave(128, -2)[..., :n, :].repeat_interleave(128, -1)[..., :k]
    return q.float() * s


def _weight8(g, lead: int, n: int, k: int):
    """E4M3 codes [lead][n][k] of a random weight, and its block scales."""
    q = torch.empty((lead, n, k), dtype=_E4M3, device="cuda")
    s = torch.empty((lead, _up(n, 128) // 128, _up(k, 128) // 128), device="cuda")
    for i in range(lead):
        q[i], s[i] = _quantize_blocks(torch.randn((n, k), generator=g, device="cuda") * 0.02)
    return q, s


def _swizzle(device) -> torch.Tensor:
    """[16][4]: which block of row r stands at position p."""
    r = torch.arange(16, device=device).unsqueeze(1)
    return torch.arange(4, device=device).unsqueeze(0) ^ ((r >> 2) & 3)


def _weight4(g, lead: int, n: int, k: int):
    """FP4 tiles [lead][kt][rt][1024] of a random weight, and their scale words."""
    rows, kt = _up(n, 16), _up(k, 128) // 128
    rt, kg = rows // 16, -(-kt // 4)
    q = torch.empty((lead, kt, rt, 1024), dtype=torch.uint8, device="cuda")
    s = torch.empty((lead, kg, rt, 64), dtype=torch.int32, device="cuda")
    at = _swizzle(q.device)
    for i in range(lead):
        w = torch.zeros((rows, kt * 128), device="cuda")
        w[:n, :k] = torch.randn((n, k), generator=g, device="cuda") * 0.02
        b = w.reshape(rows, kt * 4, 32)
        top = b.abs().amax(dim=2)
        e = torch.where(top == 0, torch.full_like(top, -127).int(), torch.frexp(top)[1] - 3)
        v = torch.ldexp(b, -e.unsqueeze(2)).abs()
        code = ((v > 0.25).to(torch.uint8) + (v >= 0.75) + (v > 1.25) + (v >= 1.75) + (v > 2.5) + (v >= 3.5) + (v > 5.0))
        code = code.to(torch.uint8) | (torch.signbit(b).to(torch.uint8) << 3)
        byte = (code[..., 0::2] | (code[..., 1::2] << 4)).reshape(rt, 16, kt, 4, 16).movedim(2, 0)
        q[i] = torch.gather(byte, 3, at.view(16, 4, 1).expand_as(byte)).reshape(kt, rt, 1024)
        eb = torch.zeros((rows, kg * 16), dtype=torch.uint8, device="cuda")
        eb[:, :kt * 4] = (e + 127).to(torch.uint8)
        eb = eb.reshape(rt, 16, kg, 4, 4).movedim(2, 0).transpose(3, 4).contiguous()  # [kg, rt, 16, b, t]
        s[i] = eb.reshape(kg, rt, 256).view(torch.int32)
    return q, s


def _plain_values4(q: torch.Tensor, scale: torch.Tensor) -> torch.Tensor:
    """FP4 tiles and scale words -> fp32 values [..][rows][k], padding included."""
    lead, (kt, rt), kg = q.shape[:-3], q.shape[-3:-1], scale.shape[-3]
    b = q.reshape(*lead, kt, rt, 16, 4, 16)
    at = _swizzle(q.device)
    b = torch.gather(b, -2, at.view(16, 4, 1).expand_as(b)).movedim(-5, -3)  # [.., rt, 16, kt, 4, 16]
    mag = torch.tensor(_MAGNITUDES, device=q.device)
    table = torch.cat((mag, -mag))
    v = table[torch.stack((b & 15, b >> 4), dim=-1).int()].reshape(*lead, rt * 16, kt * 4, 32)
    e = scale.contiguous().view(torch.uint8).reshape(*lead, kg, rt, 16, 4, 4).transpose(-1, -2).movedim(-5, -3)
    e = e.reshape(*lead, rt * 16, kg * 16)[..., :kt * 4].int() - 127
    return torch.ldexp(v, e.unsqueeze(-1)).reshape(*lead, rt * 16, kt * 128)


def _sizes(case) -> list[int]:
    """The numbers of elements of an optimizer case's tensors: a few large ones, most of them odd, many small ones."""
    rng = random.Random(case["numel"] * 31 + case["tensors"])
    share = [rng.random() ** 3 + 0.001 for _ in range(case["tensors"])]
    return [max(1, int(case["numel"] * x / sum(share))) for x in share]


def _hyper(case) -> dict:
    return {"step": case["step"], "lr": 1e-4, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.1}


def _mix(x: torch.Tensor) -> torch.Tensor:
    """The 32-bit mixing step of the optimizer's random numbers, on int64 values below 2^32."""
    x = ((x ^ (x >> 16)) * 0x9E3779B9) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0x6A09E667) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _act(name: str, g: torch.Tensor) -> torch.Tensor:
    if name == "silu":
        return g / (1.0 + torch.exp(-g))
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))


def _act_slope(name: str, g: torch.Tensor) -> torch.Tensor:
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return s * (1.0 + g * (1.0 - s))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g)


# ----------------------------------------------------------------- prepare

def prepare(case, seed):
    op = case["op"]
    g = _gen(seed)
    s = {"case": case}
    if op in ("gated", "ffn"):
        s["a"], s["a_scale"] = _plain_quantize_rows(_activation(g, case["m"], case["k"]))
        s["b"], s["b_scale"] = _weight8(g, 2, case["n"], case["k"])
        if op == "ffn":
            s["d"], s["d_scale"] = _quantize_blocks(torch.randn((case["k"], case["n"]), generator=g, device="cuda") * 0.02)
    elif op == "experts":
        _prepare_experts(s, case, seed, g)
    elif op == "backward":
        s["dh"] = (_activation(g, case["m"], case["n"]) * 1e-3).to(torch.bfloat16)
        s["gate_up"] = (_activation(g, case["m"], 2 * case["n"]) * 1.5).to(torch.bfloat16)
    elif op == "gemv":
        experts = case.get("experts", 0)
        s["x"] = _activation(g, case["m"], case["k"]).to(torch.bfloat16)
        per = 2 if case["gated"] else 1
        q, scale = _weight4(g, max(experts, 1) * per, case["n"], case["k"])
        shape = ((experts,) if experts else ()) + ((2,) if per == 2 else ())
        s["w"], s["w_scale"] = q.reshape(*shape, *q.shape[1:]), scale.reshape(*shape, *scale.shape[1:])
        if experts:
            pick = torch.rand((case["m"], experts), generator=g, device="cuda")
            s["ids"] = torch.topk(pick, case["topk"], dim=1).indices.to(torch.int32).contiguous()
    else:
        _prepare_adamw(s, case, seed, g)
    return s


def _prepare_experts(s, case, seed, g):
    rng = np.random.default_rng([seed, 21])
    popularity = np.arange(1, case["experts"] + 1) ** -case["skew"]
    rows = rng.multinomial(case["rows"], popularity[rng.permutation(case["experts"])] / popularity.sum())
    off = np.concatenate([[0], np.cumsum(-(-rows // 128) * 128)])
    # the rows that a program sets aside before it knows the routing; what is left of them is the last expert's padding
    m_total = _up(case["rows"] + case["experts"] * 127, 128)
    off[-1] = m_total
    s["offsets"] = torch.from_numpy(off.astype(np.int32)).cuda()
    s["rows"] = torch.from_numpy(rows.astype(np.int32)).cuda()
    x = _activation(g, m_total, case["k"])
    s["a"], s["a_scale"] = _plain_quantize_rows(x)
    q, scale = _weight8(g, 2 * case["experts"], case["n"], case["k"])
    s["b"], s["b_scale"] = q.reshape(-1, 2, *q.shape[1:]), scale.reshape(-1, 2, *scale.shape[1:])
    s["cap"] = int(max(rows.max(), 1))


def _prepare_adamw(s, case, seed, g):
    """Flat buffers whose tensors start on multiples of 128 elements; what lies between them is zero."""
    sizes = _sizes(case)
    padded = [_up(n, 128) for n in sizes]
    total = sum(padded)
    start = np.concatenate([[0], np.cumsum(padded)]).astype(np.int64)
    live = torch.zeros((total,), dtype=torch.bool, device="cuda")
    for at, n in zip(start, sizes):
        live[at:at + n] = True
    zero = torch.zeros((), device="cuda")

    def fill(scale):
        return torch.where(live, torch.randn((total,), generator=g, device="cuda") * scale, zero)

    s["p"] = fill(0.02)
    s["copy"] = s["p"].to(torch.bfloat16)
    size = 1e-3 * torch.exp(fill(1.0))  # elements of different sizes of gradient
    s["g"] = (fill(1.0) * size).to(torch.bfloat16)
    m, r = fill(0.3) * size, fill(0.2).abs() * size
    if case["bits"] == 8:
        for name, x in (("m", m), ("r", r)):
            b = x.reshape(-1, 128)
            sc = b.abs().amax(dim=1) / 448.0
            s[name] = (b / torch.where(sc > 0, sc, torch.ones_like(sc)).unsqueeze(1)).reshape(-1).to(_E4M3)
            s[name + "_scale"] = sc
    else:
        s["m"], s["v"] = m, r * r
    s["sizes"], s["start"] = sizes, start
    s["seed"] = seed & 0x7FFFFFFF
    views = {}
    for name in ("p", "copy", "g", "m", "r", "v"):
        if name in s:
            views[name] = [s[name][at:at + n] for at, n in zip(start, sizes)]
    for name in ("m_scale", "r_scale"):
        if name in s:
            views[name] = [s[name][at // 128:at // 128 + _up(n, 128) // 128] for at, n in zip(start, sizes)]
    s["views"] = views
    if own:
        import fine_grained_fp8_quantize_amd as fq

        s["plan"] = fq.adamw_plan(views["p"], views["m"], views["r"] if case["bits"] == 8 else views["v"],
                                  views.get("m_scale"), views.get("r_scale"), views["copy"])


# --------------------------------------------------------------------- run

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import fine_grained_fp8_quantize_amd as fq

    c = s["case"]
    op = c["op"]
    if op == "gated":
        keep = torch.empty((c["m"], 2 * c["n"]), dtype=torch.bfloat16, device="cuda") if c["keep"] else None
        h = fq.fp8_gated_gemm(s["a"], s["a_scale"], s["b"], s["b_scale"], c["act"], gate_up=keep)
        return (h, keep) if c["keep"] else h
    if op == "ffn":
        keep = torch.empty((c["m"], 2 * c["n"]), dtype=torch.bfloat16, device="cuda")
        h, h_scale = fq.fp8_gated_gemm(s["a"], s["a_scale"], s["b"], s["b_scale"], c["act"], _E4M3, gate_up=keep)
        return fq.fp8_gemm(h, h_scale, s["d"], s["d_scale"], "block", torch.bfloat16), keep
    if op == "experts":
        return fq.fp8_grouped_gated_gemm(s["offsets"], s["rows"], s["a"], s["a_scale"], s["b"], s["b_scale"], c["act"])
    if op == "backward":
        return fq.fp8_gated_backward(s["dh"], s["gate_up"], c["act"], transposed=c["transposed"])
    if op == "gemv":
        if c["gated"]:
            return fq.fp4_gated_gemv_mx(s["x"], s["w"], s["w_scale"], c["n"], c["act"], s.get("ids"),
                                        out_dtype=_dtype(c["out"]))
        return fq.fp4_gemv_mx(s["x"], s["w"], s["w_scale"], c["n"], s.get("ids"), out_dtype=_dtype(c["out"]))
    fq.adamw_step(s["plan"], s["views"]["g"], seed=s["seed"], **_hyper(c))
    return _adamw_outputs(s)


def _adamw_outputs(s):
    names = ("p", "copy", "m", "m_scale", "r", "r_scale") if s["case"]["bits"] == 8 else ("p", "copy", "m", "v")
    return {name: s[name] for name in names}


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op in ("gated", "ffn"):
        a, b = _plain_rows(s["a"], s["a_scale"]), _plain_blocks(s["b"], s["b_scale"])
        gate, up = torch.matmul(a, b[0].t()), torch.matmul(a, b[1].t())
        h = _act(c["act"], gate) * up
        keep = torch.cat((gate, up), dim=1).to(torch.bfloat16) if op == "ffn" or c["keep"] else None
        if op == "ffn":
            hq = _plain_rows(*_plain_quantize_rows(h))
            return torch.matmul(hq, _plain_blocks(s["d"], s["d_scale"]).t()).to(torch.bfloat16), keep
        return (h.to(torch.bfloat16), keep) if c["keep"] else h.to(torch.bfloat16)
    if op == "experts":
        return _plain_experts(s)
    if op == "backward":
        return _plain_backward(s)
    if op == "gemv":
        return _plain_gemv(s)
    return _plain_adamw(s)


def _plain_experts(s):
    """Every expert's rows gathered into one batch of equal heights, two batched products, the rows put back."""
    c = s["case"]
    a, b = _plain_rows(s["a"], s["a_scale"]), _plain_blocks(s["b"], s["b_scale"])
    off, rows = s["offsets"].long(), s["rows"].long()
    place = torch.arange(s["cap"], device=a.device).unsqueeze(0)
    x = a[torch.clamp(off[:-1].unsqueeze(1) + place, max=a.shape[0] - 1)]
    gate = torch.bmm(x, b[:, 0].transpose(1, 2).contiguous())
    up = torch.bmm(x, b[:, 1].transpose(1, 2).contiguous())
    y = _act(c["act"], gate) * up
    r = torch.arange(a.shape[0], device=a.device)
    e = torch.clamp(torch.searchsorted(off, r, right=True) - 1, max=c["experts"] - 1)
    i = r - off[e]
    out = y[e, torch.clamp(i, max=s["cap"] - 1)]
    return torch.where((i < rows[e]).unsqueeze(1), out, torch.zeros_like(out)).to(torch.bfloat16)


def _plain_backward(s):
    c = s["case"]
    n = c["n"]
    dh, gate, up = s["dh"].float(), s["gate_up"][:, :n].float(), s["gate_up"][:, n:].float()
    d = torch.cat((dh * up * _act_slope(c["act"], gate), dh * _act(c["act"], gate)), dim=1)
    q = _plain_quantize_rows(d)
    return (*q, *_plain_quantize_rows(d.t())) if c["transposed"] else q


def _plain_gemv(s):
    c = s["case"]
    x = s["x"].float()
    w = _plain_values4(s["w"], s["w_scale"])[..., :c["n"], :c["k"]]
    if "ids" in s:
        # every expert's product of every token, then the chosen ones
        y = torch.matmul(x, w.transpose(-1, -2).contiguous())  # [E, (2,) m, n]
        token = torch.arange(c["m"], device=x.device).unsqueeze(1)
        y = y[s["ids"].long(), :, token] if c["gated"] else y[s["ids"].long(), token]
    else:
        y = torch.matmul(x, w.transpose(-1, -2).contiguous())
        y = y.movedim(0, 1) if c["gated"] else y
    if c["gated"]:
        y = _act(c["act"], y[..., 0, :]) * y[..., 1, :]
    return y.to(_dtype(c["out"]))


def _random_bits(s) -> torch.Tensor:
    """The 32 random bits of every element, [blocks][128]."""
    dev = s["p"].device
    blocks = torch.tensor([_up(n, 128) // 128 for n in s["sizes"]], device=dev)
    tensor = torch.repeat_interleave(torch.arange(len(s["sizes"]), device=dev), blocks)
    first = torch.repeat_interleave(torch.cumsum(blocks, 0) - blocks, blocks)
    key = _mix(torch.full((1,), s["seed"], dtype=torch.int64, device=dev))  # (the seed's upper half is zero)
    key = _mix((_mix(key) + s["case"]["step"]) & 0xFFFFFFFF)
    key = _mix(_mix((key + tensor) & 0xFFFFFFFF))  # (elements' upper halves are zero)
    at = (torch.arange(len(tensor), device=dev) - first).unsqueeze(1) * 128 + torch.arange(128, device=dev)
    return _mix(at ^ key.unsqueeze(1))


def _plain_stochastic(y: torch.Tensor, bits: torch.Tensor) -> torch.Tensor:
    """E4M3 magnitude codes of y in [0, 448], rounded up where 16 random bits pass what is cut off."""
    raw = y.view(torch.int32).long()
    normal = ((raw + (bits << 4)) >> 20) - (120 << 3)
    small = ((y * 2.0 ** 29).long() + (bits << 4)) >> 20
    return torch.clamp(torch.where(y >= 2.0 ** -6, normal, small), max=126)


def _plain_adamw(s):
    c, h = s["case"], _hyper(s["case"])
    b1, b2, t = h["beta1"], h["beta2"], h["step"]
    step_size = h["lr"] / (1.0 - b1 ** t)
    root = 1.0 / math.sqrt(1.0 - b2 ** t)
    g = s["g"].float()
    if c["bits"] == 8:
        m = (s["m"].float().reshape(-1, 128) * s["m_scale"].unsqueeze(1)).reshape(-1)
        r = (s["r"].float().reshape(-1, 128) * s["r_scale"].unsqueeze(1)).reshape(-1)
        v = r * r
    else:
        m, v = s["m"], s["v"]
    m = m * b1 + g * (1.0 - b1)
    v = v * b2 + (g * g) * (1.0 - b2)
    r = torch.sqrt(v)
    p = s["p"] * (1.0 - h["lr"] * h["weight_decay"]) - (m / (r * root + h["eps"])) * step_size
    s["p"].copy_(p)
    s["copy"].copy_(p)
    if c["bits"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return _adamw_outputs(s)
    bits = _random_bits(s)
    for name, x, half in (("m", m, bits & 0xFFFF), ("r", r, bits >> 16)):
        b = x.reshape(-1, 128)
        sc = b.abs().amax(dim=1) / 448.0
        y = b.abs() / torch.where(sc > 0, sc, torch.ones_like(sc)).unsqueeze(1)
        code = _plain_stochastic(torch.clamp(y, max=448.0), half)
        if name == "r":
            code = torch.where((b > 0) & (code == 0), torch.ones_like(code), code)
        code = code | (torch.signbit(b).long() << 7)
        s[name].copy_(code.to(torch.uint8).reshape(-1).view(_E4M3))
        s[name + "_scale"].copy_(sc)
    return _adamw_outputs(s)


# -------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op in ("gated", "ffn"):
        m, n, k = case["m"], case["n"], case["k"]
        b, f = (m + 2 * n) * k + m * k / 32, 4.0 * m * n * k
        if op == "gated":
            return {"bytes": b + m * n * (6.0 if case["keep"] else 2.0), "flops": f}
        return {"bytes": b + m * n * 4.0 + n * k + 2.0 * m * k, "flops": f + 2.0 * m * n * k}
    if op == "experts":
        m, n, k, e = case["rows"], case["n"], case["k"], min(case["experts"], case["rows"])
        return {"bytes": (m + 2.0 * e * n) * k + m * k / 32 + 2.0 * m * n, "flops": 4.0 * m * n * k}
    if op == "backward":
        e = case["m"] * case["n"]
        return {"bytes": e * (10.0 if case["transposed"] else 8.0), "flops": 30.0 * e}
    if op == "gemv":
        m, n, k = case["m"], case["n"], case["k"]
        routes, per = m * case.get("topk", 1), 2 if case["gated"] else 1
        read = min(case["experts"], routes) if "experts" in case else 1
        return {"bytes": read * per * n * k * 17.0 / 32 + 2.0 * m * k + routes * n * (2 if case["out"] == "bf16" else 4),
                "flops": 2.0 * routes * per * n * k}
    n = sum(_sizes(case))
    return {"bytes": n * (12.0 + (16.0 if case["bits"] == 32 else 4.0 + 16.0 / 128)), "flops": 20.0 * n}


# ------------------------------------------------------------------- exact

def _exact_codes(codes: torch.Tensor) -> torch.Tensor:
    """The values of E4M3 codes, from their bits, in 64 bits."""
    c = codes.view(torch.uint8).long()
    e, f = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e == 0, f * 2.0 ** -9, (8.0 + f) * torch.exp2((e - 10).double()))
    return torch.where(c >= 128, -mag, mag)


def _exact_matrix(q, scale, rows: int, cols: int) -> torch.Tensor:
    """Codes [r][c] times the scale that stands for `rows` x `cols` of them."""
    r = torch.arange(q.shape[0], device=q.device) // rows
    c = torch.arange(q.shape[1], device=q.device) // cols
    return _exact_codes(q) * scale.double()[r.unsqueeze(1), c.unsqueeze(0)]


def _exact_act(name: str, g: torch.Tensor):
    """act(g) and its slope."""
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * torch.sigmoid(-g)
    c = math.sqrt(2.0 / math.pi)
    z = 2.0 * c * (g + 0.044715 * g ** 3)
    s = torch.sigmoid(z)  # (1 + tanh(z / 2)) / 2
    return g * s, s + g * s * torch.sigmoid(-z) * 2.0 * c * (1.0 + 0.134145 * g * g)


def _exact_round(y: torch.Tensor) -> torch.Tensor:
    """|y| <= 448 rounded to the E4M3 grid, ties to even."""
    _, e = torch.frexp(y)
    step = torch.exp2((torch.clamp(e, min=-5) - 4).double())
    return torch.round(y / step) * step


def _exact_tiles(x: torch.Tensor):
    """[rows][cols] -> values of the codes in 1x128 tiles, scales [cols/128][rows]."""
    t = x.reshape(x.shape[0], -1, 128)
    s = t.abs().amax(dim=2, keepdim=True) / 448.0
    y = _exact_round(torch.where(s > 0, t / torch.where(s > 0, s, 1.0), torch.zeros_like(t)))
    return y.reshape(x.shape), s.squeeze(2).t()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("gated", "ffn"):
        a = _exact_matrix(s["a"], s["a_scale"].t(), 1, 128)
        gate = torch.matmul(a, _exact_matrix(s["b"][0], s["b_scale"][0], 128, 128).t().contiguous())
        up = torch.matmul(a, _exact_matrix(s["b"][1], s["b_scale"][1], 128, 128).t().contiguous())
        h = _exact_act(case["act"], gate)[0] * up
        if op == "gated":
            return (h, torch.cat((gate, up), 1)) if case["keep"] else h
        y, scale = _exact_tiles(h)
        hq = y * scale.t().repeat_interleave(128, 1)
        down = _exact_matrix(s["d"], s["d_scale"], 128, 128)
        return torch.matmul(hq, down.t().contiguous()), torch.cat((gate, up), 1)
    if op == "experts":
        out = torch.zeros((s["a"].shape[0], case["n"]), dtype=torch.float64, device="cuda")
        off, rows = s["offsets"].cpu().tolist(), s["rows"].cpu().tolist()
        for e in range(case["experts"]):
            if rows[e]:
                at = slice(off[e], off[e] + rows[e])
                a = _exact_matrix(s["a"][at], s["a_scale"][:, at].t(), 1, 128)
                gate, up = (torch.matmul(a, _exact_matrix(s["b"][e, i], s["b_scale"][e, i], 128, 128).t().contiguous())
                            for i in (0, 1))
                out[at] = _exact_act(case["act"], gate)[0] * up
        return out
    if op == "backward":
        n = case["n"]
        dh, gate, up = s["dh"].double(), s["gate_up"][:, :n].double(), s["gate_up"][:, n:].double()
        act, slope = _exact_act(case["act"], gate)
        d = torch.cat((dh * up * slope, dh * act), dim=1)
        return (*_exact_tiles(d), *_exact_tiles(d.t().contiguous())) if case["transposed"] else _exact_tiles(d)
    if op == "gemv":
        return _exact_gemv(s)
    return _exact_adamw(s)


def _exact_matrix4(q: torch.Tensor, scale: torch.Tensor) -> torch.Tensor:
    """FP4 tiles [kt][rt][1024] -> float64 [rows][k], element by element from the layout's formula."""
    kt, rt = q.shape[0], q.shape[1]
    r = torch.arange(rt * 16, device=q.device).unsqueeze(1)
    k = torch.arange(kt * 128, device=q.device).unsqueeze(0)
    block = (k % 128) // 32
    byte = (r % 16) * 64 + (block ^ ((r % 16) // 4)) * 16 + (k % 32) // 2
    code = (q[k // 128, r // 16, byte].int() >> (4 * (k % 2))) & 15
    word = scale[k // 512, r // 16, (r % 16) * 4 + block]
    e = (word >> (8 * ((k // 128) % 4))) & 255
    m, x = code & 1, (code >> 1) & 3
    mag = torch.where(x == 0, 0.5 * m, (1.0 + 0.5 * m) * torch.exp2((x - 1).double()))
    return torch.where(code >= 8, -mag, mag).double() * torch.exp2(e.double() - 127.0)


def _exact_gemv(s):
    c = s["case"]
    n, k = c["n"], c["k"]
    x = s["x"].double()
    per = 2 if c["gated"] else 1
    w, scale = s["w"].reshape(-1, *s["w"].shape[-3:]), s["w_scale"].reshape(-1, *s["w_scale"].shape[-3:])
    ids = s["ids"].long() if "ids" in s else torch.zeros((c["m"], 1), dtype=torch.int64, device="cuda")
    out = torch.zeros((*ids.shape, n), dtype=torch.float64, device="cuda")
    for e in sorted(set(ids.reshape(-1).tolist())):
        token, place = torch.nonzero(ids == e, as_tuple=True)
        y = [torch.matmul(x[token], _exact_matrix4(w[e * per + i], scale[e * per + i])[:n, :k].t().contiguous())
             for i in range(per)]
        out[token, place] = _exact_act(c["act"], y[0])[0] * y[1] if per == 2 else y[0]
    return out if "ids" in s else out[:, 0]


def _exact_adamw(s):
    c, h = s["case"], _hyper(s["case"])
    b1, b2 = h["beta1"], h["beta2"]
    g, p = s["g"].double(), s["p"].double()
    if c["bits"] == 8:
        tile = torch.arange(len(g), device=g.device) // 128
        m = _exact_codes(s["m"]) * s["m_scale"].double()[tile]
        v = (_exact_codes(s["r"]) * s["r_scale"].double()[tile]) ** 2
    else:
        m, v = s["m"].double(), s["v"].double()
    m = b1 * m + (1.0 - b1) * g
    v = b2 * v + (1.0 - b2) * g ** 2
    first, second = m / (1.0 - b1 ** c["step"]), v / (1.0 - b2 ** c["step"])
    p = p - h["lr"] * (h["weight_decay"] * p + first / (torch.sqrt(second) + h["eps"]))
    if c["bits"] == 32:
        return {"p": p, "copy": p, "m": m, "v": v}
    bits = _random_bits(s).reshape(-1)
    got = {"p": p, "copy": p}
    for name, x, u in (("m", m, bits & 0xFFFF), ("r", torch.sqrt(v), bits >> 16)):
        scale = x.reshape(-1, 128).abs().amax(dim=1) / 448.0
        full = scale[tile]
        y = torch.where(full > 0, x.abs() / torch.where(full > 0, full, 1.0), torch.zeros_like(x))
        _, e = torch.frexp(y)
        step = torch.exp2((torch.clamp(e, min=-5) - 4).double())
        below = torch.floor(y / step)
        up = y / step - below + u.double() / 65536.0 >= 1.0
        y = torch.clamp((below + up) * step, max=448.0)
        if name == "r":
            y = torch.where((x > 0) & (y == 0), 2.0 ** -9, y)
        got[name], got[name + "_scale"] = torch.copysign(y, x), scale
    return got
