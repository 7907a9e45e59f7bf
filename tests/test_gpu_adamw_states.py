"""The AdamW step's states bit for bit, in tensors of many blocks and at the ends of fp32's range.

Every operation on the states is rounded to fp32 by itself, so its formulas taken
step by step in fp32 give the same bits, in 8 bits the same codes and scales.  New
parameters are compared with 64 bits under the bounds of test_gpu_adamw.py.
"""
from __future__ import annotations

import pytest
import torch

import software_pipelined_tiled_gemm_gb300 as sg
from tests.test_gpu_adamw import BLOCK, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    sg.check_operators()
    torch.cuda.empty_cache()


def steps_of(case, betas=(0.9, 0.999), scale=1.0):
    """The state after a step, each operation in fp32: (exp_avg, exp_avg_sq, scales)."""
    def f32(v):
        return torch.tensor(v, dtype=torch.float64).to(torch.float32).cuda()

    state, t = case.state, int(case.state.step) + 1
    total = state.exp_avg.numel()
    g = torch.zeros(total, device="cuda")
    for t_g, at in zip(case.grads, case.at):
        g[at:at + t_g.numel()] = t_g.reshape(-1).float()
    m, v = state.exp_avg.float(), state.exp_avg_sq.float()
    if state.scales is not None:
        m = m * state.scales[0].repeat_interleave(BLOCK)
        v = v * state.scales[1].repeat_interleave(BLOCK)
        v = v * v
    g = g * f32(scale)
    m = f32(betas[0]) * m + f32(1.0 - betas[0]) * g
    v = f32(betas[1]) * v + f32(1.0 - betas[1]) * (g * g)
    inside = torch.zeros(total, dtype=torch.bool, device="cuda")
    for p, at in zip(case.params, case.at):
        inside[at:at + p.numel()] = True
    m, v = torch.where(inside, m, 0.0), torch.where(inside, v, 0.0)
    if state.scales is None:
        return m, v, None
    r = v.sqrt()
    scales = torch.stack([m.abs().view(-1, BLOCK).amax(1), r.view(-1, BLOCK).amax(1)]) * f32(1.0 / 448.0)
    scales = scales.clamp(min=2.0 ** -120)
    over = (1.0 / scales).repeat_interleave(BLOCK, 1)
    # Twenty bits of fp32 are a step of e4m3, once its exponent is e4m3's.
    bits = ((r * over[1]) * 2.0 ** -120).view(torch.int32).long()
    j = torch.arange(total, device="cuda")
    codes = (bits + (((j * 0xC13FA9A9 + t * 0x91E10DA5) % 2 ** 32) >> 12)) >> 20
    codes = torch.where(r > 0, codes.clamp(1, 0x7e), 0)
    return (m * over[0]).to(torch.float8_e4m3fn), codes.to(torch.uint8).view(torch.float8_e4m3fn), scales


def bits_of(t):
    return t.view(torch.uint8 if t.dtype == torch.float8_e4m3fn else torch.int32)


def step_and_compare(case, **kw):
    want, t = case.want(1e-2, **kw)
    states = steps_of(case, **{k: v for k, v in kw.items() if k in ("betas", "scale")})
    if "scale" in kw:
        kw["scale"] = torch.tensor(kw["scale"], device="cuda")
    sg.adamw(case.params, case.grads, case.state, 1e-2, copies=case.copies, **kw)
    for name, got, expect in zip(("exp_avg", "exp_avg_sq", "scales"), case.state[1:], states):
        if expect is not None:
            # (0 in fp32 may be -0)
            same = (bits_of(got) == bits_of(expect)) | ((got.float() == 0) & (expect.float() == 0))
            assert bool(same.all()), (name, int((~same).sum()), int((~same).reshape(-1).nonzero()[0]))
    for i, (p, w) in enumerate(zip(case.params, want)):
        for name, got in [("p", p)] + ([("copy", case.copies[i])] if case.copies else []):
            value, bound = w[name]
            err = (got.double().reshape(-1) - value).abs()
            assert bool((err <= bound).all()), (i, name, float((err / bound).max()))
    assert int(case.state.step) == t


@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("bits,million", [(8, 8), (8, 16), (8, 20), (32, 12), (32, 20)])
def test_several_blocks_a_warp(bits, million, odd):
    """A warp takes a second block of a chunk from some 7.5 million elements on with 8-bit states, from
    10 million on with 32-bit ones: the ring goes round, and the last chunk of the tensor is a part of one."""
    shapes = [(300,), (million << 20,), ((1 << 20) + 777,), (1000,), (257, 3)]
    case = Case(shapes, grad="bf16", copy="bf16", bits=bits, seed=million, odd=odd)
    case.state.step.fill_(6)
    step_and_compare(case, scale=0.75)
    step_and_compare(case)


@pytest.mark.parametrize("param,grad,copy", [("bf16", "bf16", None), ("f16", "f32", "bf16"), ("f32", "f16", "f16")])
def test_several_blocks_a_warp_of_other_types(param, grad, copy):
    step_and_compare(Case([(17 << 20,), (5,)], param, grad, copy, 8, seed=1))
    step_and_compare(Case([(11 << 20,), (5,)], param, grad, copy, 32, seed=2))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-22, 1e-17, 1e6, 1e15])
def test_gradients_of_any_size(bits, size):
    case = Case([(600,), (5,)], copy="f16", bits=bits, seed=6, size=size)
    case.state = sg.adamw_state(case.params, bits)
    for _ in range(3):
        step_and_compare(case, eps=0.0 if size > 1 else 1e-8)


def test_all_of_the_state_repeats():
    """Scales too: eagerly, on another stream and in a graph that is replayed."""
    a, b, c = (Case([(5000,), (1 << 21,), (31, 9)], grad="bf16", copy="bf16", bits=8, seed=9) for _ in range(3))

    def step(case):
        sg.adamw(case.params, case.grads, case.state, 1e-2, copies=case.copies)
    step(c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i in range(4):
        step(a)
        with torch.cuda.stream(side):
            step(b)
        if i:
            graph.replay()
    torch.cuda.synchronize()
    for other in (b, c):
        assert int(other.state.step) == 4
        for x, y in zip(a.params + a.copies + list(a.state[1:]), other.params + other.copies + list(other.state[1:])):
            assert torch.equal(x.float(), y.float())


@pytest.mark.parametrize("bits", [32, 8])
def test_eps_at_the_ends_of_the_range(bits):
    """An eps whose reciprocal fp32 does not hold is refused; the least one leaves a parameter without gradients as it was."""
    case = Case([(300,)], bits=bits, seed=3)
    case.state = sg.adamw_state(case.params, bits)
    for eps in (1e-39, 1e-50, 1e38, 1e300, float("inf"), float("nan"), -1e-8):
        with pytest.raises(sg.GemmError, match="eps"):
            sg.adamw(case.params, case.grads, case.state, 1e-2, eps=eps)
    assert int(case.state.step) == 0
    before, g = case.params[0].clone(), [torch.zeros_like(case.grads[0])]
    for eps in (2.0 ** -126, 2.0 ** 126):
        sg.adamw(case.params, g, case.state, 1e-2, eps=eps, weight_decay=0.0)
        assert torch.equal(case.params[0], before)
