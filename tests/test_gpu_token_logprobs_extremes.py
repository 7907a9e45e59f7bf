"""Log probabilities and their gradient where logits are large, masked with
finite values or not numbers, on the GPU against the definition in 64 bits.

Tolerances are those of test_gpu_token_logprobs.py, which hold for logits of
any size: log p is the difference of a logit and the row's largest (one
rounding of its value) less ln s, and lse the sum of that largest and ln s
(one rounding).
"""
from __future__ import annotations

import math

import pytest
import torch

import software_pipelined_tiled_gemm_gb300 as sg
from tests.test_gpu_token_logprobs import DT, INF, close

pytestmark = pytest.mark.gpu

# One row shared by a cluster, a few rows, and more rows than blocks.
SHAPES = [(1, 70001), (3, 2600), (900, 2600)]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    sg.check_operators()


def reference(logits, tokens, k):
    """The definition in 64 bits, every difference from the row's largest logit
    taken first: beyond 2^53 even 64 bits lose ln s beside it."""
    x = logits.double().cpu()
    m = x.amax(1, keepdim=True)
    log_s = torch.logsumexp(x - m, 1, keepdim=True)
    lp = (x - m) - log_s
    p = lp.exp()
    out = {"lse": (m + log_s)[:, 0], "entropy": -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(1), "p": p,
           "lp": lp, "logprobs": lp.gather(1, tokens.cpu()[:, None])[:, 0]}
    if k:
        out["top_ids"] = x.sort(dim=1, descending=True, stable=True).indices[:, :k]
        out["top_logprobs"] = lp.gather(1, out["top_ids"])
    return out


def check(logits, tokens, k):
    r = sg.token_logprobs(logits, tokens, top_k=k)
    want = reference(logits, tokens, k)
    for name in ("lse", "entropy", "logprobs") + (("top_logprobs",) if k else ()):
        close(getattr(r, name), want[name], name)
    if k:
        assert torch.equal(r.top_ids.cpu(), want["top_ids"])
    return r, want


def normal(t, v, seed):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(t, v, generator=gen) * 3, torch.randint(0, v, (t,), generator=gen).cuda()


@pytest.mark.parametrize("t,v", SHAPES, ids=str)
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_log_probabilities_of_columns_masked_with_the_lowest_value(dt, t, v):
    x, tokens = normal(t, v, seed=4)
    low = torch.finfo(DT[dt]).min
    y = x.to(DT[dt])
    y[:, 4:] = low                # fewer possible columns than alternatives
    tokens[:] = v - 2
    r, want = check(y.cuda(), tokens, 8)
    assert (r.logprobs == torch.finfo(DT[dt]).min).all() if dt != "f16" else torch.isfinite(r.logprobs).all()
    assert torch.isfinite(r.top_logprobs).all() and r.top_ids[:, 4:].tolist() == [[4, 5, 6, 7]] * t


@pytest.mark.parametrize("t,v", SHAPES, ids=str)
@pytest.mark.parametrize("mask", [-1e4, -4e6, -5e6, -1e10, -3e9, -1e12, -1e20, -1e30, -3e38])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_columns_masked_with_a_large_negative_value(dt, mask, t, v):
    x, tokens = normal(t, v, seed=1)
    tokens.clamp_(max=v // 2 - 1)
    for columns in (slice(0, v // 3), slice(v // 2, v), slice(0, v, 2), slice(0, 0)):
        y = x.clone()
        y[:, columns] = mask
        y = y.to(DT[dt]).cuda()
        for k in (0, 6):
            check(y, tokens, k)


@pytest.mark.parametrize("t,v", SHAPES, ids=str)
@pytest.mark.parametrize("mask", [-1e4, -4e6, -5e6, -1e10, -3e9, -1e12, -1e20, -1e30, -3e38])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_a_row_of_one_large_negative_value_is_uniform(dt, mask, t, v):
    y = torch.full((t, v), mask).to(DT[dt]).cuda()
    tokens = torch.full((t,), 5, device="cuda")
    for k in (0, 6):
        r, _ = check(y, tokens, k)
        assert (r.logprobs + math.log(v)).abs().max() < 1e-5
        assert (r.entropy - math.log(v)).abs().max() < 1e-4


@pytest.mark.parametrize("t,v", SHAPES, ids=str)
@pytest.mark.parametrize("offset", [1e4, 1e6, 3.9e6, 4.1e6, 1.7e7, 1e10, 1e20, 1e38, -1e4, -1e6, -4.1944e6, -1e10, -1e20])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_rows_far_from_zero(dt, offset, t, v):
    x, tokens = normal(t, v, seed=2)
    y = (x + offset).to(DT[dt]).cuda()
    y[:, v // 3] = offset - 4     # between rows' values wherever the type resolves it
    for k in (0, 6):
        check(y, tokens, k)


@pytest.mark.parametrize("t,v", SHAPES, ids=str)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_rows_across_the_whole_range(dt, t, v):
    # Each thread meets elements of every size, the largest of them last or first.
    x, tokens = normal(t, v, seed=3)
    size = 10.0 ** (torch.arange(v) * 7919 % 38).float()
    for sign in (-1.0, 1.0):
        y = (x.abs() * sign * size).to(DT[dt]).cuda()
        for k in (0, 6):
            check(y, tokens, k)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("t,v,k", [(1, 1, 1), (1, 20, 20), (600, 20, 20), (1, 131072, 64), (2, 2600, 5), (700, 2600, 33)])
def test_nan_ranks_first_from_the_first_column_on(dt, t, v, k):
    nan = float("nan")
    x, _ = normal(t, v, seed=8)
    for columns in ([0], [0, v - 1], list(range(v))):
        y = x.clone()
        y[:, columns] = nan
        y = y.to(DT[dt])
        if v > 2:
            y[:, 1] = nan if len(columns) == v else -INF
        r = sg.token_logprobs(y.cuda(), None, top_k=k)
        want = (y.float() + 0.0).sort(dim=1, descending=True, stable=True).indices[:, :k]
        assert torch.equal(r.top_ids.cpu(), want)
        assert torch.isnan(r.lse).all() and torch.isnan(r.entropy).all()
        picked = y.float().gather(1, want)
        assert (torch.isnan(r.top_logprobs.cpu()) == (picked != -INF)).all()
        assert (r.top_logprobs.cpu()[picked == -INF] == -INF).all()


def gradient_within_bounds(x, tokens, dt):
    """The gradient against its formula, and its sum over each row."""
    t, v = x.shape
    r, want = check(x, tokens, 0)
    gen = torch.Generator().manual_seed(5)
    gl, gh = torch.randn(t, generator=gen), torch.randn(t, generator=gen)
    p, lp = want["p"], want["lp"]
    plp = torch.where(p > 0, p * lp, torch.zeros_like(p))
    for a, b in ((gl, gh), (gl, None), (None, gh)):
        d = sg.token_logprobs_backward(x, tokens, r, None if a is None else a.cuda(),
                                       None if b is None else b.cuda()).double().cpu()
        l64 = (torch.zeros(t) if a is None else a).double()
        h64 = (torch.zeros(t) if b is None else b).double()
        exact = -l64[:, None] * p - h64[:, None] * (plp + p * want["entropy"][:, None])
        exact[torch.arange(t), tokens.cpu()] += l64
        # As in test_gpu_token_logprobs.py, plus the roundings of g and g_H (x - p) themselves.
        tol = 2.0 ** -18 * (l64.abs()[:, None] * (p + (p > 0.5))
                            + h64.abs()[:, None] * (plp.abs() + p * (want["entropy"] + 13)[:, None])) + 1e-30
        u = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dt]
        tol = tol + u * (exact.abs() + tol) + (2.0 ** -24 if dt == "f16" else 1e-38)
        assert ((d - exact).abs() <= tol).all(), float(((d - exact).abs() / tol).max())
        assert (d.sum(1).abs() <= tol.sum(1) + exact.sum(1).abs()).all()


@pytest.mark.parametrize("t,v", SHAPES, ids=str)
@pytest.mark.parametrize("value", ["lowest", "highest", -1e30, -1e10, -5e6, 1e4, 1e6, 1e10, 1e30])
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_gradient_of_rows_of_one_value(dt, value, t, v):
    info = torch.finfo(DT[dt])
    value = {"lowest": info.min, "highest": info.max}.get(value, value)
    if abs(value) > info.max:
        pytest.skip("beyond the type")
    x = torch.full((t, v), value).to(DT[dt]).cuda()
    gradient_within_bounds(x, torch.full((t,), v // 2, device="cuda"), dt)


@pytest.mark.parametrize("t,v", SHAPES, ids=str)
@pytest.mark.parametrize("offset", [1e4, -1e4, 1e6, -1e6, 1e7])
def test_gradient_of_rows_far_from_zero(offset, t, v):
    x, tokens = normal(t, v, seed=6)
    gradient_within_bounds((x + offset).cuda(), tokens, "f32")


def test_a_result_without_the_low_part_is_taken():
    # Five fields, lse alone: as precise as fp32 holds it.
    x, tokens = normal(7, 1000, seed=7)
    r, want = check(x.cuda(), tokens, 0)
    g = torch.rand(7, generator=torch.Generator().manual_seed(8))
    old = sg.TokenLogprobs(*r[:5])
    a = sg.token_logprobs_backward(x.cuda(), tokens, r, g.cuda(), g.cuda()).double().cpu()
    b = sg.token_logprobs_backward(x.cuda(), tokens, old, g.cuda(), g.cuda()).double().cpu()
    # lse (below 16) rounds within 2^-21, log p L (below 30) within 2^-20 of p's value either way
    p, lp, h, g = want["p"], want["lp"].abs(), want["entropy"][:, None], g.double()[:, None]
    assert ((a - b).abs() <= 2.0 ** -17 * g * p * (2 + lp + h) + 2.0 ** -23 * a.abs() + 1e-30).all()
