"""Workloads of the 4-bit microscaling operators and of the MoE routing operators.

``listed()`` names the cases, ``draw()`` makes more of the same ranges,
``prepare()`` builds a case's inputs on the GPU, ``run()`` makes one pass: in
plain torch operations where ``own`` is false, through the package where it is
true. ``exact()`` gives the same outputs in 64 bits.

FP4 matrices are held in tiles of 16 rows x 128 k (1 KB): ``q`` is uint8
``[kt][rt][1024]``, row r of a tile at byte 64 r and its 32-element block b (16
bytes, low nibble first) at 16 * (b ^ ((r >> 2) & 3)) inside the row; ``scale``
is int32 ``[ceil(kt/4)][rt][64]``, word 4 r + b holding the E8M0 bytes of block
b of four consecutive k tiles.
"""
from __future__ import annotations

import random

import numpy as np
import torch

own = False

_MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases

def listed():
    return [
        # a dense layer's activations, quantized along their channels and read back
        {"name": "quant_rows_4096x7168", "op": "quantize", "rows": 4096, "cols": 7168, "tiling": "1x32"},
        # the token-contiguous operand of a weight gradient, an odd channel count
        {"name": "quant_tokens_8192x2040", "op": "quantize", "rows": 8192, "cols": 2040, "tiling": "32x1"},
        # tokens quantized once and sent to the rows of the local experts
        {"name": "quant_scatter_8192x7168", "op": "scatter", "tokens": 8192, "cols": 7168, "topk": 8,
         "experts": 256, "first": 32, "local": 32, "align": 128},
        # one token through a layer: every weight read for one row of output
        {"name": "gemm_decode_1x4096x7168", "op": "gemm", "m": 1, "n": 4096, "k": 7168, "out": "bf16"},
        # a small batch, odd sizes, fp32 output
        {"name": "gemm_batch_131x2050x7136", "op": "gemm", "m": 131, "n": 2050, "k": 7136, "out": "f32"},
        # a dense layer in training or prefill
        {"name": "gemm_4096x4096x7168", "op": "gemm", "m": 4096, "n": 4096, "k": 7168, "out": "bf16"},
        # serving: 16 tokens over 32 experts, one or a few rows each, some none
        {"name": "experts_decode_32x2048x4096", "op": "grouped", "tokens": 16, "topk": 4, "experts": 32, "n": 2048,
         "k": 4096, "align": 16, "skew": 0.0, "out": "bf16"},
        # training: 8192 routed rows over 32 experts of uneven popularity
        {"name": "experts_8192x4096x7168", "op": "grouped", "tokens": 1024, "topk": 8, "experts": 32, "n": 4096,
         "k": 7168, "align": 128, "skew": 1.1, "out": "bf16"},
        # the balance loss of a small step, bf16 logits, sigmoid scores
        {"name": "balance_96x32", "op": "balance", "tokens": 96, "experts": 32, "topk": 4, "seqs": 3,
         "score": "sigmoid", "dtype": "bf16"},
        # the balance loss of a training step, per sequence, softmax scores
        {"name": "balance_16384x256", "op": "balance", "tokens": 16384, "experts": 256, "topk": 8, "seqs": 4,
         "score": "softmax", "dtype": "f32"},
        # the row layout of a serving step
        {"name": "dispatch_64x32", "op": "dispatch", "tokens": 64, "topk": 4, "experts": 32, "first": 0, "local": 32,
         "align": 16},
        # the row layout of a training step, one rank's share of the experts
        {"name": "dispatch_16384x256", "op": "dispatch", "tokens": 16384, "topk": 8, "experts": 256, "first": 0,
         "local": 256, "align": 128},
    ]


def _log_int(rng: random.Random, lo: int, hi: int) -> int:
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng: random.Random):
    op = rng.choice(["quantize", "scatter", "gemm", "gemm", "grouped", "grouped", "balance", "dispatch"])
    if op == "quantize":
        return {"op": op, "rows": _log_int(rng, 1, 4096), "cols": _log_int(rng, 32, 7168),
                "tiling": rng.choice(["1x32", "32x1"])}
    if op == "scatter":
        experts = rng.choice([8, 32, 64, 256])
        local = max(1, experts // rng.choice([1, 4, 8]))
        topk = rng.randint(1, 8)
        return {"op": op, "tokens": _log_int(rng, 1, 8192 * local // (experts * topk) + 1024),
                "cols": _log_int(rng, 32, 7168), "topk": topk, "experts": experts,
                "first": rng.randint(0, experts - local), "local": local, "align": rng.choice([16, 128])}
    if op == "gemm":
        return {"op": op, "m": _log_int(rng, 1, 4096), "n": _log_int(rng, 16, 4096), "k": _log_int(rng, 32, 7168),
                "out": rng.choice(["bf16", "f32"])}
    if op == "grouped":
        experts = rng.choice([4, 8, 31, 32])
        return {"op": op, "tokens": _log_int(rng, 1, 1024), "topk": rng.randint(1, min(8, experts)),
                "experts": experts, "n": _log_int(rng, 64, 4096), "k": _log_int(rng, 64, 7168),
                "align": rng.choice([16, 128]), "skew": rng.choice([0.0, 0.6, 1.1]),
                "out": rng.choice(["bf16", "f32"])}
    if op == "balance":
        experts = rng.choice([8, 20, 64, 160, 256])
        return {"op": op, "tokens": _log_int(rng, 1, 16384), "experts": experts,
                "topk": rng.randint(1, 8), "seqs": _log_int(rng, 1, 8), "score": rng.choice(["softmax", "sigmoid"]),
                "dtype": rng.choice(["bf16", "f32"])}
    experts = rng.choice([8, 20, 64, 256])
    local = max(1, experts // rng.choice([1, 4]))
    return {"op": op, "tokens": _log_int(rng, 1, 16384), "topk": rng.randint(1, 8), "experts": experts,
            "first": rng.randint(0, experts - local), "local": local, "align": rng.choice([16, 128])}


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
    """N(0, 1) with one entry in a thousand fifty times larger, as bf16."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    big = torch.rand((rows, cols), generator=g, device="cuda") < 1e-3
    return torch.where(big, x * 50.0, x).to(torch.bfloat16)


def _weight(g, *shape) -> torch.Tensor:
    return (torch.randn(shape, generator=g, device="cuda") * 0.02).to(torch.bfloat16)


def _block_codes(x: torch.Tensor):
    """E2M1 codes [..][nb][32] and biased exponents [..][nb] of blocks of 32."""
    amax = x.abs().amax(dim=-1)
    e = torch.clamp(torch.frexp(amax)[1] - 3, -127, 127)
    e = torch.where(amax == 0, torch.full_like(e, -127), e)
    v = torch.ldexp(x, -e.unsqueeze(-1)).abs()
    # between two neighbours the nearer one; a tie goes to the even code
    code = ((v > 0.25).to(torch.uint8) + (v >= 0.75) + (v > 1.25) + (v >= 1.75) + (v > 2.5) + (v >= 3.5) + (v > 5.0))
    return code.to(torch.uint8) | (torch.signbit(x).to(torch.uint8) << 3), e + 127


def _swizzle(device) -> torch.Tensor:
    """[16][4]: which block of row r stands at position p."""
    r = torch.arange(16, device=device).unsqueeze(1)
    return torch.arange(4, device=device).unsqueeze(0) ^ ((r >> 2) & 3)


def _to_tiles(codes: torch.Tensor, ebytes: torch.Tensor):
    """codes [.., rows, nb, 32], ebytes [.., rows, nb] (rows % 16 == 0, nb % 4 == 0) -> q, scale tiles."""
    lead = codes.shape[:-3]
    rows, nb = codes.shape[-3], codes.shape[-2]
    kt, rt = nb // 4, rows // 16
    b = codes[..., 0::2] | (codes[..., 1::2] << 4)
    b = b.reshape(*lead, rt, 16, kt, 4, 16).movedim(-3, -5)          # [.., kt, rt, 16, 4, 16]
    at = _swizzle(codes.device)
    q = torch.gather(b, -2, at.view(16, 4, 1).expand_as(b)).reshape(*lead, kt, rt, 1024).contiguous()
    kg = -(-kt // 4)
    e = torch.zeros((*lead, rows, kg * 16), dtype=torch.uint8, device=codes.device)
    e[..., :nb] = ebytes.to(torch.uint8)
    e = e.reshape(*lead, rt, 16, kg, 4, 4).movedim(-3, -5).transpose(-1, -2)  # [.., kg, rt, 16, b, t]
    s = e.contiguous().reshape(*lead, kg, rt, 256).view(torch.int32)
    return q, s


def _plain_quantize(x: torch.Tensor):
    """[.., rows, cols] -> q, scale tiles, blocks along the last dimension."""
    rows, cols = x.shape[-2:]
    p = torch.nn.functional.pad(x.float(), (0, _up(cols, 128) - cols, 0, _up(rows, 16) - rows))
    codes, e = _block_codes(p.reshape(*p.shape[:-1], -1, 32))
    return _to_tiles(codes, e)


def _plain_codes(q: torch.Tensor, scale: torch.Tensor):
    """q, scale tiles -> codes [.., rows, nb, 32] and biased exponents [.., rows, nb]."""
    lead = q.shape[:-3]
    kt, rt = q.shape[-3], q.shape[-2]
    b = q.reshape(*lead, kt, rt, 16, 4, 16)
    at = _swizzle(q.device)
    b = torch.gather(b, -2, at.view(16, 4, 1).expand_as(b)).movedim(-5, -3)  # [.., rt, 16, kt, 4, 16]
    codes = torch.stack((b & 15, b >> 4), dim=-1).reshape(*lead, rt * 16, kt * 4, 32)
    kg = scale.shape[-3]
    e = scale.contiguous().view(torch.uint8).reshape(*lead, kg, rt, 16, 4, 4).transpose(-1, -2).movedim(-5, -3)
    return codes, e.reshape(*lead, rt * 16, kg * 16)[..., :kt * 4]


def _plain_values(q: torch.Tensor, scale: torch.Tensor) -> torch.Tensor:
    """q, scale tiles -> fp32 values [.., rows, k], padding included."""
    codes, e = _plain_codes(q, scale)
    mag = torch.tensor(_MAGNITUDES, device=q.device)
    table = torch.cat((mag, -mag))
    v = torch.ldexp(table[codes.int()], (e.int() - 127).unsqueeze(-1))
    return v.reshape(*v.shape[:-2], -1)


def _plain_plan(ids: torch.Tensor, first: int, local: int, align: int):
    """group_offsets, group_rows, dst_rows of expert ids [tokens][topk]."""
    flat = ids.reshape(-1).long() - first
    hot = torch.arange(local, device=ids.device).unsqueeze(1) == flat.unsqueeze(0)
    upto = torch.cumsum(hot.to(torch.int32), dim=1, dtype=torch.int32)
    rows = upto[:, -1].contiguous()
    padded = (rows + align - 1) // align * align
    off = torch.nn.functional.pad(torch.cumsum(padded, 0, dtype=torch.int32), (1, 0))
    here = (flat >= 0) & (flat < local)
    e = torch.clamp(flat, 0, local - 1)
    dst = off[e] + torch.gather(upto, 0, e.unsqueeze(0)).squeeze(0) - 1
    dst = torch.where(here, dst, torch.full_like(dst, -1))
    return off, rows, dst.reshape(ids.shape).to(torch.int32)


def _ids(seed: int, tokens: int, topk: int, experts: int, skew: float) -> np.ndarray:
    """Distinct experts of each token, expert popularity (rank + 1)^-skew in a random order."""
    rng = np.random.default_rng([seed, 11])
    topk = min(topk, experts)
    logp = -skew * np.log(np.arange(1, experts + 1))[rng.permutation(experts)]
    score = logp + rng.gumbel(size=(tokens, experts))
    return np.argsort(-score, axis=1, kind="stable")[:, :topk].astype(np.int32)


def _capacity(case, share: float) -> int:
    """Rows a program sets aside for an expert-sorted layout before it knows the routing."""
    local = case.get("local", case["experts"])
    routes = case["tokens"] * min(case["topk"], case["experts"])
    return _up(min(routes, int(routes * share) + 16) + local * (case["align"] - 1), case["align"])


# ----------------------------------------------------------------- prepare

def prepare(case, seed):
    op = case["op"]
    g = _gen(seed)
    s = {"case": case}
    if op == "quantize":
        s["x"] = _activation(g, case["rows"], case["cols"])
    elif op == "scatter":
        ids = torch.from_numpy(_ids(seed, case["tokens"], case["topk"], case["experts"], 0.5)).cuda()
        s["x"] = _activation(g, case["tokens"], case["cols"])
        s["dst"] = _plain_plan(ids, case["first"], case["local"], case["align"])[2]
        # (routes past the rows set aside are dropped)
        s["m_total"] = _capacity(case, 1.5 * case["local"] / case["experts"])
        kt = -(-case["cols"] // 128)
        s["q"] = torch.zeros((kt, s["m_total"] // 16, 1024), dtype=torch.uint8, device="cuda")
        s["scale"] = torch.zeros((-(-kt // 4), s["m_total"] // 16, 64), dtype=torch.int32, device="cuda")
    elif op == "gemm":
        s["a"], s["a_scale"] = _plain_quantize(_activation(g, case["m"], case["k"]))
        s["b"], s["b_scale"] = _plain_quantize(_weight(g, case["n"], case["k"]))
    elif op == "grouped":
        ids = torch.from_numpy(_ids(seed, case["tokens"], case["topk"], case["experts"], case["skew"])).cuda()
        off, rows, dst = _plain_plan(ids, 0, case["experts"], case["align"])
        s["offsets"], s["rows"] = off, rows
        m_total = _capacity(case, 1.0)
        x = _activation(g, case["tokens"], case["k"])
        sorted_x = torch.zeros((m_total, case["k"]), dtype=torch.bfloat16, device="cuda")
        sorted_x[dst.reshape(-1).long()] = x.repeat_interleave(ids.shape[1], 0)
        s["a"], s["a_scale"] = _plain_quantize(sorted_x)
        s["b"], s["b_scale"] = _plain_quantize(_weight(g, case["experts"], case["n"], case["k"]))
        s["cap"] = int(rows.max())
    elif op == "balance":
        t, e = case["tokens"], case["experts"]
        bias = 0.5 * torch.randn((1, e), generator=g, device="cuda")
        logits = torch.randn((t, e), generator=g, device="cuda") + bias
        s["logits"] = logits.to(_dtype(case["dtype"]))
        ids = torch.topk(s["logits"].float(), min(case["topk"], e), dim=1).indices.to(torch.int32)
        # the last tokens of the batch are padding; a few routes were dropped
        ids[t - t // 16:] = -1
        dropped = torch.rand(ids.shape, generator=g, device="cuda") < 0.01
        s["ids"] = torch.where(dropped, torch.full_like(ids, -1), ids).contiguous()
        rng = np.random.default_rng([seed, 12])
        cuts = np.sort(rng.integers(0, t + 1, case["seqs"] - 1))
        s["seq_offsets"] = torch.from_numpy(np.concatenate([[0], cuts, [t]]).astype(np.int32)).cuda()
        s["grad"] = torch.rand((1,), generator=g, device="cuda") + 0.5
    else:
        s["ids"] = torch.from_numpy(_ids(seed, case["tokens"], case["topk"], case["experts"], 0.8)).cuda()
    return s


# --------------------------------------------------------------------- run

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import fine_grained_fp8_quantize_amd as fq

    c = s["case"]
    op = c["op"]
    if op == "quantize":
        q, scale = fq.fp4_quantize_mx(s["x"], c["tiling"])
        rows, cols = (c["rows"], c["cols"]) if c["tiling"] == "1x32" else (c["cols"], c["rows"])
        return fq.fp4_dequantize_mx(q, scale, rows, cols)
    if op == "scatter":
        fq.fp4_quantize_mx_scatter(s["x"], s["dst"], s["m_total"], q=s["q"], scale=s["scale"])
        return fq.fp4_dequantize_mx(s["q"], s["scale"], s["m_total"], c["cols"])
    if op == "gemm":
        return fq.fp4_gemm_mx(s["a"], s["a_scale"], s["b"], s["b_scale"], c["m"], c["n"], _dtype(c["out"]))
    if op == "grouped":
        return fq.fp4_grouped_gemm_mx(s["offsets"], s["rows"], s["a"], s["a_scale"], s["b"], s["b_scale"], c["n"],
                                      _dtype(c["out"]))
    if op == "balance":
        loss, counts, coef = fq.moe_balance_loss(s["logits"], s["ids"], s["seq_offsets"], c["score"], 0.01)
        grad = fq.moe_balance_loss_backward(s["logits"], s["ids"], coef, s["grad"], s["seq_offsets"], c["score"])
        return loss, counts, grad
    return fq.moe_dispatch(s["ids"], c["local"], c["align"], c["first"])


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "quantize":
        x = s["x"] if c["tiling"] == "1x32" else s["x"].t()
        q, scale = _plain_quantize(x)
        return _plain_values(q, scale)[:x.shape[0], :x.shape[1]].to(torch.bfloat16)
    if op == "scatter":
        return _plain_scatter(s)
    if op == "gemm":
        a, b = _plain_values(s["a"], s["a_scale"]), _plain_values(s["b"], s["b_scale"])
        return torch.matmul(a[:c["m"]], b[:c["n"]].t()).to(_dtype(c["out"]))
    if op == "grouped":
        return _plain_grouped(s)
    if op == "balance":
        return _plain_balance(s)
    return _plain_plan(s["ids"], c["first"], c["local"], c["align"])


def _plain_scatter(s):
    """Codes of every token, then the rows of q that the routes name."""
    x, dst = s["x"], s["dst"]
    cols = x.shape[1]
    codes, e = _block_codes(torch.nn.functional.pad(x.float(), (0, _up(cols, 128) - cols)).reshape(len(x), -1, 32))
    old_codes, old_e = _plain_codes(s["q"], s["scale"])
    # routes to nowhere write a row past the end
    to = torch.where((dst < 0) | (dst >= s["m_total"]), torch.full_like(dst, s["m_total"]), dst).reshape(-1).long()
    new_codes = torch.cat((old_codes, old_codes[:1])).index_copy(0, to, codes.repeat_interleave(dst.shape[1], 0))[:-1]
    new_e = torch.cat((old_e, old_e[:1])).index_copy(0, to, e.to(torch.uint8).repeat_interleave(dst.shape[1], 0))[:-1]
    q, scale = _to_tiles(new_codes, new_e)
    return _plain_values(q, scale)[:, :cols].to(torch.bfloat16)


def _plain_grouped(s):
    """Every expert's rows gathered into one batch of equal heights, one batched product, the rows put back."""
    c = s["case"]
    a = _plain_values(s["a"], s["a_scale"])
    b = _plain_values(s["b"], s["b_scale"])[:, :c["n"]]
    off, rows = s["offsets"].long(), s["rows"].long()
    place = torch.arange(s["cap"], device=a.device).unsqueeze(0)
    src = torch.clamp(off[:-1].unsqueeze(1) + place, max=a.shape[0] - 1)
    y = torch.bmm(a[src], b.transpose(1, 2).contiguous())
    r = torch.arange(a.shape[0], device=a.device)
    e = torch.clamp(torch.searchsorted(off, r, right=True) - 1, max=c["experts"] - 1)
    i = r - off[e]
    real = (i < rows[e]).unsqueeze(1)
    out = y[e, torch.clamp(i, max=s["cap"] - 1)]
    return torch.where(real, out, torch.zeros_like(out)).to(_dtype(c["out"]))


def _plain_balance(s):
    c = s["case"]
    x, ids = s["logits"].float(), s["ids"]
    experts, seqs = c["experts"], s["seq_offsets"].numel() - 1
    u = x if c["score"] == "softmax" else -torch.log1p(torch.exp(-x))
    ex = torch.exp(u - u.amax(dim=1, keepdim=True))
    p = ex / ex.sum(dim=1, keepdim=True)
    token = torch.arange(x.shape[0], device=x.device)
    seq = torch.searchsorted(s["seq_offsets"][1:].contiguous(), token.int(), right=True)
    in_seq = (seq.unsqueeze(0) == torch.arange(seqs, device=x.device).unsqueeze(1))          # [seqs][tokens]
    valid = (ids >= 0) & (ids < experts)
    hot = ((ids.unsqueeze(2) == torch.arange(experts, device=x.device)) & valid.unsqueeze(2)).sum(dim=1)
    counted = valid.any(dim=1)
    counts = torch.zeros((seqs, experts), dtype=torch.int64, device=x.device).index_add(0, seq, hot)
    used = (in_seq & counted.unsqueeze(0)).float()
    tokens = used.sum(dim=1)
    live = (tokens > 0).float()
    freq = experts * counts.float() / torch.clamp(counts.sum(dim=1, keepdim=True).float(), min=1.0)
    mean = torch.matmul(used, p) / torch.clamp(tokens, min=1.0).unsqueeze(1)
    nlive = torch.clamp(live.sum(), min=1.0)
    loss = 0.01 * (freq * mean).sum() / nlive
    coef = 0.01 * freq / (torch.clamp(tokens, min=1.0) * nlive).unsqueeze(1)
    w = coef[seq]
    du = s["grad"] * p * (w - (p * w).sum(dim=1, keepdim=True))
    if c["score"] == "sigmoid":
        du = du / (1.0 + torch.exp(x))
    du = torch.where(counted.unsqueeze(1), du, torch.zeros_like(du))
    return loss.reshape(1), counts.to(torch.int32), du.to(s["logits"].dtype)


# -------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    codes = 0.5 + 1.0 / 32.0  # bytes of an element's code and of its share of a scale
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": 4.0 * n, "flops": 2.0 * n}
    if op == "scatter":
        routed = case["tokens"] * case["topk"] * case["local"] / case["experts"]
        return {"bytes": 2.0 * case["cols"] * (case["tokens"] + routed), "flops": 2.0 * case["tokens"] * case["cols"]}
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m + n) * k * codes + m * n * (2 if case["out"] == "bf16" else 4), "flops": 2.0 * m * n * k}
    if op == "grouped":
        rows = case["tokens"] * min(case["topk"], case["experts"])
        experts, n, k = min(case["experts"], rows), case["n"], case["k"]
        return {"bytes": (rows + experts * n) * k * codes + rows * n * (2 if case["out"] == "bf16" else 4),
                "flops": 2.0 * rows * n * k}
    if op == "balance":
        n = case["tokens"] * case["experts"]
        return {"bytes": n * 2.0 * (2 if case["dtype"] == "bf16" else 4) + 4.0 * case["tokens"] * case["topk"],
                "flops": 12.0 * n}
    return {"bytes": 8.0 * case["tokens"] * case["topk"] + 8.0 * case["local"],
            "flops": 2.0 * case["tokens"] * case["topk"]}


# ------------------------------------------------------------------- exact

def _exact_rounded(x: torch.Tensor) -> torch.Tensor:
    """Every value of [rows][cols] replaced by what its block of 32 stores for it, in 64 bits."""
    rows, cols = x.shape
    b = torch.zeros((rows, _up(cols, 32)), dtype=torch.float64, device=x.device)
    b[:, :cols] = x
    b = b.view(rows, -1, 32)
    top = b.abs().amax(dim=2, keepdim=True)
    e = torch.floor(torch.log2(torch.where(top > 0, top, torch.full_like(top, 2.0 ** -200)))) - 2
    unit = torch.exp2(torch.clamp(e, -127, 127))
    v = torch.clamp(b.abs() / unit, max=6.0)
    # spacing of the grid: 0.5 below 2, 1 below 4, 2 up to 6; a tie goes to the even multiple, which is the even code
    step = torch.where(v < 2, 0.5, torch.where(v < 4, 1.0, 2.0)).double()
    v = torch.round(v / step) * step
    return (torch.copysign(v, b) * unit).view(rows, -1)[:, :cols]


def _exact_values(q: torch.Tensor, scale: torch.Tensor) -> torch.Tensor:
    """q [kt][rt][1024], scale -> float64 [rows][k], element by element from the layout's formula."""
    kt, rt = q.shape[0], q.shape[1]
    r = torch.arange(rt * 16, device=q.device).unsqueeze(1)
    k = torch.arange(kt * 128, device=q.device).unsqueeze(0)
    block = (k % 128) // 32
    byte = (r % 16) * 64 + (block ^ ((r % 16) // 4)) * 16 + (k % 32) // 2
    code = (q[k // 128, r // 16, byte].int() >> (4 * (k % 2))) & 15
    word = scale[k // 512, r // 16, (r % 16) * 4 + block]
    e = (word >> (8 * ((k // 128) % 4))) & 255
    m = code & 1
    x = (code >> 1) & 3
    mag = torch.where(x == 0, 0.5 * m, (1.0 + 0.5 * m) * torch.exp2((x - 1).double()))
    return torch.where(code >= 8, -mag, mag).double() * torch.exp2(e.double() - 127.0)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = s["x"].double()
        return _exact_rounded(x if case["tiling"] == "1x32" else x.t())
    if op == "scatter":
        v = _exact_rounded(s["x"].double())
        out = torch.zeros((s["m_total"], case["cols"]), dtype=torch.float64, device=v.device)
        dst = s["dst"].long()
        for k in range(dst.shape[1]):
            here = (dst[:, k] >= 0) & (dst[:, k] < s["m_total"])
            out[dst[here, k]] = v[here]
        return out
    if op == "gemm":
        a, b = _exact_values(s["a"], s["a_scale"])[:case["m"]], _exact_values(s["b"], s["b_scale"])[:case["n"]]
        return torch.matmul(a, b.t().contiguous())
    if op == "grouped":
        a = _exact_values(s["a"], s["a_scale"])
        out = torch.zeros((a.shape[0], case["n"]), dtype=torch.float64, device=a.device)
        off, rows = s["offsets"].cpu().tolist(), s["rows"].cpu().tolist()
        for e in range(case["experts"]):
            if rows[e]:
                b = _exact_values(s["b"][e], s["b_scale"][e])[:case["n"]]
                out[off[e]:off[e] + rows[e]] = torch.matmul(a[off[e]:off[e] + rows[e]], b.t().contiguous())
        return out
    if op == "balance":
        x = s["logits"].double().cpu().numpy()
        ids, cut = s["ids"].cpu().numpy(), s["seq_offsets"].cpu().numpy()
        counted = ((ids >= 0) & (ids < case["experts"])).any(axis=1)
        seqs = [np.flatnonzero(counted[a:b]) + a for a, b in zip(cut[:-1], cut[1:])]
        seqs = [t for t in seqs if len(t)]
        loss, grad = 0.0, np.zeros_like(x)
        for t in seqs:
            one, d = _exact_sequence(x[t], ids[t], case["score"])
            loss += one / len(seqs)
            grad[t] = float(s["grad"].cpu()[0]) * d / len(seqs)
        return np.array([loss]), None, grad
    return None


def _exact_sequence(x: np.ndarray, ids: np.ndarray, score: str):
    """The balance loss of one sequence's logits, and its gradient, both times 0.01."""
    experts = x.shape[1]
    raw = np.exp(x - x.max(axis=1, keepdims=True)) if score == "softmax" else 1.0 / (1.0 + np.exp(-x))
    p = raw / raw.sum(axis=1, keepdims=True)
    n = np.bincount(ids[(ids >= 0) & (ids < experts)], minlength=experts)
    f = 0.01 * experts * n / n.sum()
    w = f / len(x)
    d = p * (w - (p * w).sum(axis=1, keepdims=True))
    return float((f * p.mean(axis=0)).sum()), d if score == "softmax" else d * (1.0 - raw)
