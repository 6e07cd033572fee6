"""The optimizer step on the GPU: bit for bit against the float32 model, whose
step is held to the formula in float64; many tensors, odd sizes and addresses,
8-bit states, options that live on the GPU, captured steps."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fine_grained_fp8_quantize_amd as fq
from oracle import adamw as model

pytestmark = pytest.mark.gpu

HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _values(rng, n, scale):
    return (rng.standard_normal(n) * np.exp(rng.standard_normal(n)) * scale).astype(np.float32)


def _rounded(x, dt):
    """x as the values that a tensor of this type holds."""
    return x if dt == "f32" else (model.bf16(x).astype(np.uint32) << 16).view(np.float32)


def _put(x, dtype, shift):
    """x on the GPU, `shift` elements into a buffer of its own."""
    buf = torch.empty(len(x) + shift, dtype=dtype, device="cuda")
    t = buf[shift:]
    src = torch.from_numpy(x).cuda()
    t.copy_(src if dtype != torch.float8_e4m3fn else src.view(torch.float8_e4m3fn))
    return t


class Tensors:
    """A few tensors on both sides: arrays of the model, tensors of the GPU."""

    def __init__(self, sizes, param="f32", grad="bf16", bits=32, shift=0, copies=True, seed=1):
        rng = np.random.default_rng(seed)
        self.bits, self.param = bits, param
        self.p = [_rounded(_values(rng, n, 0.02), param) for n in sizes]
        self.g = [_rounded(_values(rng, n, 1e-3), grad) for n in sizes]
        m, r = [_values(rng, n, 1e-3) for n in sizes], [np.abs(_values(rng, n, 1e-3)) for n in sizes]
        self.tp = [_put(x, DT[param], shift) for x in self.p]
        self.tg = [_put(x, DT[grad], shift) for x in self.g]
        self.tc = [torch.full((n,), float("nan"), dtype=torch.bfloat16, device="cuda") for n in sizes] \
            if copies and param == "f32" else None
        if bits == 32:
            self.m, self.v = m, [x * x for x in r]
            self.tm, self.tv = ([_put(x, torch.float32, shift) for x in xs] for xs in (self.m, self.v))
            scales = ()
        else:
            zero = np.zeros
            self.mc, self.ms = zip(*[model.encode(x, zero(len(x)), False) for x in m]) if sizes else ((), ())
            self.vc, self.vs = zip(*[model.encode(x, zero(len(x)), True) for x in r]) if sizes else ((), ())
            self.mc, self.ms, self.vc, self.vs = (list(x) for x in (self.mc, self.ms, self.vc, self.vs))
            self.tm, self.tv = ([_put(x, torch.float8_e4m3fn, shift) for x in xs] for xs in (self.mc, self.vc))
            self.tms, self.tvs = ([_put(x, torch.float32, 0) for x in xs] for xs in (self.ms, self.vs))
            scales = (self.tms, self.tvs)
        self.plan = fq.adamw_plan(self.tp, self.tm, self.tv, *(scales or (None, None)), self.tc)

    def model_step(self, i, step, seed=0, grad_scale=1.0, lr=None):
        h = dict(HYPER, lr=HYPER["lr"] if lr is None else lr)
        if self.bits == 8:
            s = np.arange(len(self.p[i])) // 128
            m = model.decode_e4m3(self.mc[i]) * self.ms[i][s]
            r = model.decode_e4m3(self.vc[i]) * self.vs[i][s]
            v = r * r
        else:
            m, v = self.m[i], self.v[i]
        p, m, r, v = model.step32(self.p[i], self.g[i], m, v, step=step, grad_scale=grad_scale, **h)
        self.p[i] = _rounded(p, self.param)
        if self.bits == 8:
            bits = model.random_bits(len(p), i, step, seed)
            self.mc[i], self.ms[i] = model.encode(m, bits & np.uint64(0xFFFF), False)
            self.vc[i], self.vs[i] = model.encode(r, bits >> np.uint64(16), True)
        else:
            self.m[i], self.v[i] = m, v

    def check(self, what, copies=True):
        for i in range(len(self.p)):
            name = "%s, tensor %d of %d elements: " % (what, i, len(self.p[i]))
            pairs = [("param", self.tp[i].float(), self.p[i])]
            if self.tc is not None and copies:
                pairs.append(("copy", self.tc[i].view(torch.int16), model.bf16(self.p[i]).view(np.int16)))
            if self.bits == 8:
                pairs += [("exp_avg", self.tm[i].view(torch.uint8), self.mc[i]),
                          ("exp_avg_scale", self.tms[i], self.ms[i]),
                          ("exp_avg_sq", self.tv[i].view(torch.uint8), self.vc[i]),
                          ("exp_avg_sq_scale", self.tvs[i], self.vs[i])]
            else:
                pairs += [("exp_avg", self.tm[i], self.m[i]), ("exp_avg_sq", self.tv[i], self.v[i])]
            for part, got, want in pairs:
                got = got.cpu().numpy()
                bad = np.flatnonzero(got.view(np.uint8 if got.itemsize == 1 else "u%d" % got.itemsize)
                                     != want.view(np.uint8 if want.itemsize == 1 else "u%d" % want.itemsize))
                assert len(bad) == 0, (name + part, len(bad), bad[:4], got[bad[:4]], want[bad[:4]])


SIZES = [1, 3, 127, 128, 129, 4095, 4096, 4097, 0, 12291, 20000]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,grad", [("f32", "bf16"), ("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("shift", [0, 1, 4])
def test_steps_match_the_model(bits, param, grad, shift):
    t = Tensors(SIZES, param, grad, bits, shift)
    for step in (1, 2, 1000):
        fq.adamw_step(t.plan, t.tg, step, seed=step * 77, **HYPER)
        for i in range(len(SIZES)):
            t.model_step(i, step, seed=step * 77)
        t.check("step %d" % step)


def test_the_formula_in_64_bits():
    """Roundings of 2^-24 each: m has one of the scaled gradient, two of constants, two of products and one
    of the sum (at most 4 on either term); v 6 on its positive terms, so its root 4; the divisor 7; the update
    11 beside m's own; the parameter's two products and the difference 3."""
    n, u = 50000, 2.0 ** -24
    t = Tensors([n], "f32", "f32", 32, seed=5)
    p, g, m, v = t.p[0].copy(), t.g[0].copy(), t.m[0].copy(), t.v[0].copy()
    scale = torch.tensor([0.37], device="cuda")
    fq.adamw_step(t.plan, t.tg, 7, grad_scale=scale, **HYPER)
    s = float(scale.cpu()[0])
    want_p, want_m, want_v = model.step64(p, g, m, v, step=7, grad_scale=s, **HYPER)
    terms = np.abs(0.9 * m.astype(np.float64)) + np.abs(0.1 * s * g.astype(np.float64))
    room_m = 4.01 * u * terms
    assert np.all(np.abs(t.tm[0].cpu().numpy() - want_m) <= room_m)
    assert np.all(np.abs(t.tv[0].cpu().numpy() - want_v) <= 6.01 * u * want_v)
    divisor = (np.sqrt(want_v / (1 - 0.95 ** 7)) + 1e-8) * (1 - 0.9 ** 7) / HYPER["lr"]
    room = 3.01 * u * (np.abs(p) + terms / divisor) + (11.01 + 4.01) * u * terms / divisor
    assert np.all(np.abs(t.tp[0].cpu().numpy() - want_p) <= room)


@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_a_launch_holds(bits):
    sizes = [1 + (i * 37) % 300 for i in range(130)]
    t = Tensors(sizes, bits=bits, seed=2)
    fq.adamw_step(t.plan, t.tg, 3, seed=1 << 40, **HYPER)
    for i in range(len(sizes)):
        t.model_step(i, 3, seed=1 << 40)
    t.check("130 tensors")


@pytest.mark.parametrize("bits", [32, 8])
def test_tensors_without_a_gradient_stay(bits):
    t = Tensors([500, 600, 700], bits=bits, copies=False, seed=3)
    fq.adamw_step(t.plan, [t.tg[0], None, t.tg[2]], 2, seed=9, **HYPER)
    for i in (0, 2):
        t.model_step(i, 2, seed=9)
    t.check("one without")
    fq.adamw_step(t.plan, [None] * 3, 3, **HYPER)
    t.check("none with")
    fq.adamw_step(t.plan, [None, t.tg[1], None], 3, seed=9, **HYPER)
    t.model_step(1, 3, seed=9)
    t.check("the other one")


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_scale_that_is_not_finite_changes_nothing(value):
    for bits in (32, 8):
        t = Tensors([300, 5000], bits=bits, copies=False, seed=4)
        fq.adamw_step(t.plan, t.tg, 2, grad_scale=torch.tensor([value], device="cuda"), **HYPER)
        t.check("skipped")


@pytest.mark.parametrize("bits", [32, 8])
def test_step_and_rate_on_the_gpu_and_replays(bits):
    t = Tensors([300, 5000, 4096], bits=bits, seed=6)
    step = torch.ones(1, dtype=torch.int64, device="cuda")
    lr = torch.tensor([1e-3], device="cuda")
    scale = torch.tensor([1.0], device="cuda")
    h = {k: v for k, v in HYPER.items() if k != "lr"}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        fq.adamw_step(t.plan, t.tg, step, lr, grad_scale=scale, seed=21, **h)
    t.check("captured, not run", copies=False)
    for k in range(1, 6):
        rate, by = 1e-3 / k, 0.5 * k
        step.fill_(k)
        lr.fill_(rate)
        scale.fill_(by)
        graph.replay()
        torch.cuda.synchronize()
        for i in range(3):
            t.model_step(i, k, seed=21, grad_scale=by, lr=float(np.float32(rate)))
        t.check("replay %d" % k)


def test_a_bad_gradient_stays_in_its_block():
    for bad in (float("nan"), float("inf")):
        t = Tensors([1000], bits=8, seed=7)
        t.tg[0][300] = bad
        fq.adamw_step(t.plan, t.tg, 2, seed=3, **HYPER)
        with np.errstate(all="ignore"):
            t.model_step(0, 2, seed=3)
        m = model.decode_e4m3(t.tm[0].view(torch.uint8).cpu().numpy()) * t.tms[0].cpu().numpy()[np.arange(1000) // 128]
        assert not np.isfinite(m[256:384]).any() and np.isfinite(m[:256]).all() and np.isfinite(m[384:]).all()
        keep = np.r_[0:256, 384:1000]
        assert np.array_equal(t.tp[0].cpu().numpy()[keep], t.p[0][keep])
        assert np.array_equal(t.tm[0].view(torch.uint8).cpu().numpy()[keep], t.mc[0][keep])
        p = t.tp[0].cpu().numpy()
        assert not np.isfinite(p[300]) and np.isfinite(np.delete(p, 300)).all()


def test_rounding_is_unbiased_and_repeats():
    """An element of value c + f between neighbouring codes c, c + 1 goes up with probability f; over n elements
    the share is within 6 standard deviations, 6 sqrt(f (1 - f) / n), of it, and of 2^-16 for the random bits."""
    n = 1 << 18
    # beta1 = 0.5, m = 0: the new moment is half the gradient; the first of each block is the largest, 448
    frac = 0.3
    g = np.full(n, 2 * (20.0 + 2.0 * frac), np.float32)  # codes 20 and 22 are neighbours
    g[::128] = 2 * 448.0
    arrays = dict(p=np.zeros(n, np.float32), m=np.zeros(n, np.uint8), v=np.zeros(n, np.uint8))

    def step(seed, at):
        t = {k: torch.from_numpy(x.copy()).cuda() for k, x in arrays.items()}
        s = [torch.zeros(n // 128, device="cuda") for _ in range(2)]
        plan = fq.adamw_plan([t["p"]], [t["m"]], [t["v"]], [s[0]], [s[1]])
        fq.adamw_step(plan, [torch.from_numpy(g).cuda()], at, 1e-3, 0.5, 0.5, seed=seed)
        return t["m"].cpu().numpy(), t["v"].cpu().numpy()

    (m, v), again, other, later = step(5, 1), step(5, 1), step(6, 1), step(5, 2)
    assert np.array_equal(m, again[0]) and np.array_equal(v, again[1])
    rest = np.arange(n) % 128 != 0
    low = model.decode_e4m3(m[rest]) == 20.0
    assert np.all(low | (model.decode_e4m3(m[rest]) == 22.0))
    room = 6 * np.sqrt(frac * (1 - frac) / rest.sum()) + 2.0 ** -16
    for codes in (m, other[0], later[0]):
        assert abs((model.decode_e4m3(codes[rest]) == 22.0).mean() - frac) <= room
    for codes in (other[0], later[0]):  # independent of the first: both up with probability frac^2
        both = ((codes[rest] == m[rest]) & ~low).mean()
        assert abs(both - frac ** 2) <= 6 * np.sqrt(frac ** 2 * (1 - frac ** 2) / rest.sum()) + 2.0 ** -16


def test_a_root_above_zero_is_not_stored_as_zero():
    n = 1280
    g = np.full(n, 1e-12, np.float32)
    g[::128] = 1.0
    g[5::128] = 0.0
    t = [torch.zeros(n, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda"),
         torch.zeros(n, dtype=torch.uint8, device="cuda")]
    s = [torch.zeros(n // 128, device="cuda") for _ in range(2)]
    plan = fq.adamw_plan([t[0]], [t[1]], [t[2]], [s[0]], [s[1]])
    fq.adamw_step(plan, [torch.from_numpy(g).cuda()], 1, 1e-3)
    v = t[2].cpu().numpy()
    assert np.array_equal(v == 0, g == 0)


def test_streams_and_odd_calls():
    t, s = Tensors([40000], bits=8, seed=8), Tensors([40000], bits=8, seed=9)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for k in range(1, 4):
        for x, st in ((t, streams[0]), (s, streams[1])):
            fq.adamw_step(x.plan, x.tg, k, seed=1, stream=st, **HYPER)
    torch.cuda.synchronize()
    for x in (t, s):
        for k in range(1, 4):
            x.model_step(0, k, seed=1)
        x.check("two streams")
    empty = fq.adamw_plan([], [], [])
    fq.adamw_step(empty, [], 1, 1e-3)


def test_a_plan_keeps_its_storage():
    """A parameter that is given other storage: the plan's step changes what it was made for, which it keeps alive."""
    t = Tensors([4096, 100])
    plan = fq.adamw_plan(t.tp, t.tm, t.tv, copies=t.tc)
    before = [p.clone() for p in t.tp]
    old = t.tp[0].detach()
    t.tp[0].data = before[0].clone()
    assert t.tp[0].data_ptr() != old.data_ptr()
    del t.tm, t.tv
    fq.adamw_step(plan, t.tg, 1, **HYPER)
    assert torch.equal(t.tp[0], before[0]) and not torch.equal(old, before[0])
    assert torch.equal(t.tc[0], old.to(torch.bfloat16))


def test_refusals():
    f = lambda n, dt=torch.float32: torch.zeros(n, dtype=dt, device="cuda")  # noqa: E731
    E = fq.Fp8qError
    with pytest.raises(E, match="exp_avg has 0"):
        fq.adamw_plan([f(4)], [], [f(4)])
    with pytest.raises(E, match="dtype"):
        fq.adamw_plan([f(4)], [f(4, torch.bfloat16)], [f(4)])
    with pytest.raises(E, match="must be float32 or bfloat16"):
        fq.adamw_plan([f(4, torch.float16)], [f(4)], [f(4)])
    with pytest.raises(E, match="shape"):
        fq.adamw_plan([f(4)], [f(4)], [f(5)])
    with pytest.raises(E, match="both moments"):
        fq.adamw_plan([f(4)], [f(4, torch.uint8)], [f(4, torch.uint8)], [f(1)])
    with pytest.raises(E, match="expected \\(2,\\)"):
        fq.adamw_plan([f(129)], [f(129, torch.uint8)], [f(129, torch.uint8)], [f(1)], [f(1)])
    with pytest.raises(E, match="copies belong"):
        fq.adamw_plan([f(4, torch.bfloat16)], [f(4)], [f(4)], copies=[f(4, torch.bfloat16)])
    with pytest.raises(E, match="contiguous"):
        fq.adamw_plan([f(8)[::2]], [f(4)], [f(4)])
    with pytest.raises(E, match="share memory"):
        x = f(8)
        fq.adamw_plan([x[:4], x[2:6]], [f(4), f(4)], [f(4), f(4)])
    with pytest.raises(E, match="live on the GPU"):
        fq.adamw_plan([torch.zeros(4)], [f(4)], [f(4)])
    plan = fq.adamw_plan([f(4), f(6)], [f(4), f(6)], [f(4), f(6)])
    with pytest.raises(E, match="grads has 1"):
        fq.adamw_step(plan, [f(4)], 1, 1e-3)
    with pytest.raises(E, match="grads\\[1\\]"):
        fq.adamw_step(plan, [f(4), f(6, torch.bfloat16)], 1, 1e-3)
    with pytest.raises(E, match="grads\\[1\\]"):
        fq.adamw_step(plan, [f(4), f(4)], 1, 1e-3)
    with pytest.raises(E, match="grads\\[0\\]"):
        fq.adamw_step(plan, [torch.zeros(4), f(6)], 1, 1e-3)
    with pytest.raises(E, match="step"):
        fq.adamw_step(plan, [f(4), f(6)], 0, 1e-3)
    with pytest.raises(E, match="seed"):
        fq.adamw_step(plan, [f(4), f(6)], 1, 1e-3, seed=-1)
    with pytest.raises(E, match="lr must hold"):
        fq.adamw_step(plan, [f(4), f(6)], 1, f(2))
    with pytest.raises(E, match="step must hold"):
        fq.adamw_step(plan, [f(4), f(6)], f(1), 1e-3)
    with pytest.raises(E, match="status 2"):
        fq.adamw_step(plan, [f(4), f(6)], 1, 1e-3, beta1=1.0)
