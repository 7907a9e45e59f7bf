"""The AdamW step on the GPU against its formulas in 64 bits.

Bounds, with e = 2^-24.  m and v: each of two terms has a rounded factor and two
roundings, the sum one: 5 e of the terms' sizes.  1 - beta^t from expm1: its
argument is within 2 e, its sensitivity at most 1, the function within 2 e;
with the quotient 6 e, and half of it under the root.  The update's quotient:
these, the root's 4 e, the sum's e, 3 e of the division: below 2^-20 of it, and
what m is off.  p: four roundings of its size, and the type's.

8 bits: the codes are those of the values in 64 bits, but where a value lies so
near to a border between two codes that 2^-17 of it decide.
"""
from __future__ import annotations

import pytest
import torch

import software_pipelined_tiled_gemm_gb300 as sg

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 1e-38, torch.float16: 2.0 ** -24, torch.float32: 1e-38}
E = 2.0 ** -24
BLOCK = sg.ADAMW_BLOCK
SHAPES = [(1,), (7,), (255,), (0,), (256,), (257,), (100, 33), (64, 64), (5000,), (3, 1, 8)]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    sg.check_operators()


def starts(shapes):
    at, out = 0, []
    for s in shapes:
        out.append(at)
        at += -(-torch.Size(s).numel() // BLOCK) * BLOCK
    return out, at


def values(state):
    """(m, v) in 64 bits."""
    m, v = state.exp_avg.double(), state.exp_avg_sq.double()
    if state.scales is not None:
        s = state.scales.double().repeat_interleave(BLOCK, 1)
        m, v = m * s[0], (v * s[1]) ** 2
    return m, v


def to_codes(y, u=None):
    """The e4m3 values of y in 64 bits, and how near a border (in steps) each was."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    at = y / step
    low = torch.floor(at if u is None else at + u)
    frac = (at if u is None else at + u) - low
    if u is None:
        return torch.round(at) * step, (frac - 0.5).abs(), at.abs()
    return low * step, torch.minimum(frac, 1 - frac), at.abs()


def dither(count, t):
    j = torch.arange(count, device="cuda")
    u = (j * 0xC13FA9A9 + (t * 0x91E10DA5) % 2 ** 32) % 2 ** 32
    return (u // 4096).double() * 2.0 ** -20


class Case:
    """Random parameters, gradients and states; `odd`: addresses that allow no vectors."""

    def __init__(self, shapes, param="f32", grad="f32", copy=None, bits=32, seed=0, odd=0, size=1e-2):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def make(shape, scale, dtype):
            n = torch.Size(shape).numel()
            flat = torch.full((n + 16,), float("nan"), device="cuda", dtype=dtype)
            flat[odd:odd + n] = torch.randn(n, generator=gen, device="cuda") * scale
            return flat[odd:odd + n].view(shape)
        self.params = [make(s, 0.5, DT[param]) for s in shapes]
        self.grads = [make(s, size, DT[grad]) for s in shapes]
        self.copies = [make(s, 1.0, DT[copy]) for s in shapes] if copy else None
        self.state = sg.adamw_state(self.params, bits)
        self.at, total = starts(shapes)
        n = self.state.exp_avg.numel()
        assert n == total
        m, r = torch.randn(n, generator=gen, device="cuda"), torch.randn(n, generator=gen, device="cuda").abs() + 1e-3
        if bits == 32:
            self.state.exp_avg.copy_(m * size)
            self.state.exp_avg_sq.copy_((r * size) ** 2)
        else:
            self.state.exp_avg.copy_((m * 100).clamp(-448, 448).to(torch.float8_e4m3fn))
            self.state.exp_avg_sq.copy_((r * 100).clamp(max=448).to(torch.float8_e4m3fn))
            self.state.scales.copy_(torch.rand(2, n // BLOCK, generator=gen, device="cuda") * size / 100)

    def want(self, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, scale=1.0):
        """Per tensor {name: (value, bound)} after a step from here."""
        t = int(self.state.step) + 1
        ms, vs = values(self.state)
        decays = weight_decay if isinstance(weight_decay, list) else [weight_decay] * len(self.params)
        out = []
        for p, g, at, d in zip(self.params, self.grads, self.at, decays):
            n = p.numel()
            g = g.double().reshape(-1) * scale
            m0, v0 = ms[at:at + n], vs[at:at + n]
            m, v = betas[0] * m0 + (1 - betas[0]) * g, betas[1] * v0 + (1 - betas[1]) * g * g
            e_m = 5 * E * (betas[0] * m0.abs() + (1 - betas[0]) * g.abs()) + 1e-44
            e_v = 7 * E * v + 1e-44
            den = (v / (1 - betas[1] ** t)).sqrt() + eps
            q = lr / (1 - betas[0] ** t) * m / den
            e_q = 2.0 ** -20 * q.abs() + lr / (1 - betas[0] ** t) * e_m / den
            p0 = p.double().reshape(-1)
            new = p0 - lr * d * p0 - q
            bound = e_q + 4 * E * (p0.abs() + q.abs())
            out.append({"m": (m, e_m), "v": (v, e_v),
                        "p": (new, bound + U[p.dtype] * (new.abs() + bound) + TINY[p.dtype])})
            if self.copies is not None:
                dt = self.copies[0].dtype
                out[-1]["copy"] = (new, bound + U[dt] * (new.abs() + bound) + TINY[dt])
        return out, t

    def check(self, want, t):
        bits = 32 if self.state.scales is None else 8
        for i, (p, at, w) in enumerate(zip(self.params, self.at, want)):
            n = p.numel()
            got = {"p": p.reshape(-1)}
            if self.copies is not None:
                got["copy"] = self.copies[i].reshape(-1)
            if bits == 32:
                got["m"], got["v"] = self.state.exp_avg[at:at + n], self.state.exp_avg_sq[at:at + n]
            for name, g in got.items():
                value, bound = w[name]
                err = (g.double() - value).abs()
                assert bool((err <= bound).all()), (i, name, float((err / bound).max()))
            blocks = -(-n // BLOCK)
            pad = slice(at + n, at + blocks * BLOCK)
            assert not self.state.exp_avg[pad].float().any() and not self.state.exp_avg_sq[pad].float().any()
            if bits == 8 and n:
                full = torch.zeros(2, blocks * BLOCK, dtype=torch.float64, device="cuda")
                full[0, :n], full[1, :n] = w["m"][0], w["v"][0].sqrt()
                s = (full.abs().view(2, blocks, BLOCK).amax(2) / 448).clamp(min=2.0 ** -120)
                mine = self.state.scales[:, at // BLOCK:at // BLOCK + blocks].double()
                assert bool(((mine / s - 1).abs() <= 8 * E).all())
                y = full / s.repeat_interleave(BLOCK, 1)
                u = dither(self.state.exp_avg.numel(), t)[at:at + blocks * BLOCK]
                for k, codes in enumerate((to_codes(y[0]), to_codes(y[1], u))):
                    value, near, size = codes
                    if k == 1:
                        value = torch.where(full[1] > 0, value.clamp(min=2.0 ** -9), value)
                    value = value.clamp(-448, 448)
                    mine = (self.state.exp_avg, self.state.exp_avg_sq)[k][at:at + blocks * BLOCK].double()
                    # A step is at most 1/8 of a value, or 2^-9.
                    one = (mine - value).abs() <= value.abs() / 7 + 2.0 ** -9
                    assert bool(((mine == value) | (one & (near <= size * 2.0 ** -17))).all()), (i, k)
        assert int(self.state.step) == t


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("param,grad,copy", [("f32", "f32", None), ("f32", "bf16", "bf16"), ("f32", "f16", "f16"),
                                             ("bf16", "bf16", None), ("f16", "f32", "bf16"), ("f32", "f32", "f16")])
def test_steps(bits, odd, param, grad, copy):
    case = Case(SHAPES, param, grad, copy, bits, seed=1, odd=odd)
    case.state.step.fill_(3)
    for _ in range(3):
        want, t = case.want(1e-2)
        sg.adamw(case.params, case.grads, case.state, 1e-2, copies=case.copies)
        case.check(want, t)


@pytest.mark.parametrize("bits", [32, 8])
def test_first_step_decay_rate_and_scale(bits):
    case = Case(SHAPES, grad="bf16", copy="bf16", bits=bits, seed=2)
    case.state = sg.adamw_state(case.params, bits)
    decays = [0.1 * (i % 3) for i in range(len(SHAPES))]
    lr, scale = torch.tensor(0.03, device="cuda"), torch.tensor(0.37, device="cuda")
    args = dict(betas=(0.8, 0.95), eps=1e-6, weight_decay=decays)
    for _ in range(2):
        want, t = case.want(float(lr), scale=float(scale), **args)
        sg.adamw(case.params, case.grads, case.state, lr, copies=case.copies, scale=scale, **args)
        case.check(want, t)
    assert t == 2


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("t", [1, 1000, 123456])
def test_far_steps_and_no_momentum(bits, t):
    case = Case([(700,), (31, 9)], bits=bits, seed=3)
    case.state.step.fill_(t - 1)
    for betas in ((0.0, 0.0), (0.9, 0.9999), (0.99, 0.5)):
        want, at = case.want(1e-3, betas=betas)
        sg.adamw(case.params, case.grads, case.state, 1e-3, betas=betas)
        case.check(want, at)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("count", [33, 513, 1100])
def test_many_tensors(bits, count):
    case = Case([(1 + (i * 37) % 300,) for i in range(count)], copy="bf16", bits=bits, seed=4)
    want, t = case.want(1e-2)
    sg.adamw(case.params, case.grads, case.state, 1e-2, copies=case.copies)
    case.check(want, t)


def test_some_copies():
    case = Case([(300,), (20, 20), (5,)], copy="f16", bits=32, seed=5)
    before = case.copies[1].clone()
    want, t = case.want(1e-2)
    sg.adamw(case.params, case.grads, case.state, 1e-2, copies=[case.copies[0], None, case.copies[2]])
    assert torch.equal(case.copies[1], before)
    copies, case.copies = case.copies, None
    for w in want:
        w.pop("copy", None)
    case.check(want, t)
    assert torch.equal(copies[0], case.params[0].half()) and torch.equal(copies[2], case.params[2].half())


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("size", [1e-30, 1e-17, 1e6, 1e15])
def test_small_and_large_gradients(bits, size):
    case = Case([(600,)], bits=bits, seed=6, size=size)
    case.state = sg.adamw_state(case.params, bits)
    sg.adamw(case.params, case.grads, case.state, 1e-2, eps=0.0 if size > 1 else 1e-8, weight_decay=0.0)
    for t in (case.params[0], case.state.exp_avg.float(), case.state.exp_avg_sq.float()):
        assert bool(torch.isfinite(t).all())
    m, v = values(case.state)
    g = case.grads[0].double()
    if bits == 32:
        assert bool(((m[:600] - 0.1 * g).abs() <= 2.0 ** -22 * g.abs() + 1e-44).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_zero_gradients_leave_parameters(bits):
    case = Case([(600,), (3,)], bits=bits, seed=7)
    case.state = sg.adamw_state(case.params, bits)
    before = [p.clone() for p in case.params]
    for g in case.grads:
        g.zero_()
    for _ in range(2):
        sg.adamw(case.params, case.grads, case.state, 1e-2, weight_decay=0.0)
    assert all(torch.equal(a, b) for a, b in zip(before, case.params))
    m, v = values(case.state)
    assert not m.any() and not v.any()


@pytest.mark.parametrize("bits", [32, 8])
def test_nan_stays_in_its_element_or_block(bits):
    case = Case([(1000,), (50,)], bits=bits, seed=8)
    case.grads[0][300] = float("nan")
    case.grads[0][700] = float("inf")
    sg.adamw(case.params, case.grads, case.state, 1e-2)
    bad = torch.zeros(1000, dtype=torch.bool, device="cuda")
    bad[[300, 700]] = True
    assert torch.equal(case.params[0].isnan(), bad) and not case.params[1].isnan().any()
    m, v = values(case.state)
    if bits == 8:
        assert m[256:512].isnan().all() and m[512:768].isnan().all() and v[512:768].isnan().all()
        assert not m[:256].isnan().any() and not m[768:].isnan().any()
    else:
        assert int(m.isnan().sum()) == 1


def test_second_moment_in_8_bits_falls():
    """Half of a block's elements get no gradient any more: their v falls, which rounding to
    nearest would not let it do.

    A root moves by 5e-4 of itself a call, 0.004 steps or more of its code (a value has 8 to 16
    steps), so it falls by a step whenever the turn's fraction is below that.  Multiples of b
    come back to an interval of that length after at most 610 calls: of 0.5698, the gaps of 610
    multiples are all below 0.004.  1500 calls are two such steps at least, of a sixteenth each.
    The recursion in 64 bits with the same turns is followed element by element; an element
    may leave it where a value meets a border to within rounding, one of 1e5 values, which
    takes its root by a step of at most an eighth: below 1 % of the mean over 256 elements
    if 20 of them did.
    """
    b = 0x91E10DA5 / 2.0 ** 32
    turns = torch.sort(torch.arange(610, dtype=torch.float64) * b % 1)[0]
    assert float(torch.diff(turns, append=turns[:1] + 1).max()) < 0.004
    p = torch.zeros(512, device="cuda")
    g = torch.full((512,), 1e-3, device="cuda")
    state = sg.adamw_state([p], 8)
    v = torch.zeros(512, dtype=torch.float64, device="cuda")
    before = None
    for t in range(1, 1521):
        if t == 21:
            before = values(state)[1][::2].sqrt().mean().item()
            g[::2] = 0.0
        sg.adamw([p], [g], state, 0.0)
        root = (0.999 * v + 0.001 * g.double() ** 2).sqrt()
        s = (root.view(2, 256).amax(1) / 448).repeat_interleave(256)
        value = to_codes((root / s).clamp(max=448.0), dither(512, t))[0]
        v = (torch.where(root > 0, value.clamp(min=2.0 ** -9), value) * s) ** 2
    mine, want = values(state)[1][::2].sqrt().mean().item(), v[::2].sqrt().mean().item()
    assert mine < before * (15 / 16) ** 2
    assert abs(mine / want - 1) < 0.01, (mine, want)


def test_repeats_bit_for_bit():
    for bits in (32, 8):
        a, b = (Case(SHAPES, grad="bf16", copy="bf16", bits=bits, seed=9) for _ in range(2))
        for case in (a, b):
            for _ in range(3):
                sg.adamw(case.params, case.grads, case.state, 1e-2, copies=case.copies)
        for x, y in zip(a.params + a.copies + list(a.state[1:3]), b.params + b.copies + list(b.state[1:3])):
            assert torch.equal(x.float(), y.float())


@pytest.mark.parametrize("bits", [32, 8])
def test_streams_and_graph(bits):
    a, b = (Case(SHAPES, grad="bf16", copy="bf16", bits=bits, seed=10) for _ in range(2))
    lr = torch.tensor(1e-2, device="cuda")
    side = torch.cuda.Stream()
    for case in (a, b):     # the first step eagerly, on a stream
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            sg.adamw(case.params, case.grads, case.state, lr, copies=case.copies)
        side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sg.adamw(a.params, a.grads, a.state, lr, copies=a.copies)
    for i in range(4):      # the replays count steps and see a new rate
        lr.fill_(1e-2 / (i + 1))
        graph.replay()
        sg.adamw(b.params, b.grads, b.state, lr, copies=b.copies)
    torch.cuda.synchronize()
    assert int(a.state.step) == int(b.state.step) == 5
    for x, y in zip(a.params + a.copies + list(a.state[1:3]), b.params + b.copies + list(b.state[1:3])):
        assert torch.equal(x.float(), y.float())


def test_no_elements_still_count_the_step():
    empty = [torch.empty(0, device="cuda"), torch.empty(3, 0, device="cuda")]
    state = sg.adamw_state(empty)
    for i in range(3):
        sg.adamw(empty, empty, state, 1e-2)
        assert int(state.step) == i + 1
    # Empty tensors at the end of a list longer than a launch's table.
    case = Case([(5,)] * 512 + [(0,)] * 20, bits=32, seed=12)
    want, t = case.want(1e-2)
    sg.adamw(case.params, case.grads, case.state, 1e-2)
    case.check(want, t)


def test_refusals():
    case = Case([(300,), (20, 20)], copy="bf16", bits=8, seed=11)
    p, g, s, c = case.params, case.grads, case.state, case.copies

    def refuse(error, match, *args, **kw):
        with pytest.raises(error, match=match):
            sg.adamw(*args, **kw)
    refuse(sg.GemmError, "overlaps", [p[0], p[0]], [g[0], g[0]], sg.adamw_state([p[0], p[0]]), 1e-2)
    refuse(sg.GemmError, "overlaps", [p[0]], [p[0]], sg.adamw_state([p[0]]), 1e-2)
    refuse(sg.GemmError, "overlaps", p, g, s, 1e-2, copies=[p[1].view(torch.bfloat16).view(-1)[:300], c[1]])
    refuse(sg.GemmError, "beta", p, g, s, 1e-2, betas=(1.0, 0.9))
    refuse(sg.GemmError, "beta", p, g, s, 1e-2, betas=(0.9, float("nan")))
    refuse(sg.GemmError, "eps", p, g, s, 1e-2, eps=-1.0)
    refuse(ValueError, "length", p, g[:1], s, 1e-2)
    refuse(ValueError, "shapes", p, [g[0], g[1].view(-1)], s, 1e-2)
    refuse(ValueError, "contiguous", p, [g[0], g[1].t()], s, 1e-2)
    refuse(sg.GemmError, "state", p[:1], g[:1], s, 1e-2)
    refuse(ValueError, "state", p, g, s._replace(scales=None), 1e-2)
    refuse(ValueError, "CUDA", [p[0].cpu(), p[1]], g, s, 1e-2)
    refuse(ValueError, "lr", p, g, s, torch.tensor([1.0, 2.0], device="cuda"))
    refuse(ValueError, "scale", p, g, s, 1e-2, scale=torch.tensor(1.0, dtype=torch.float64, device="cuda"))
    refuse(ValueError, "weight_decay", p, g, s, 1e-2, weight_decay=[0.1])
    refuse(TypeError, "params", [p[0].double(), p[1]], g, s, 1e-2)
    refuse(TypeError, "copies", p, g, s, 1e-2, copies=[p[0].clone(), c[1]])
    assert int(s.step) == 0
