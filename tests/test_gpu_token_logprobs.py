"""Token log probabilities on the GPU against their definition in 64 bits.

Tolerances.  2^t by the hardware's approximation is within 2^-22, and the
sums of n positive terms by at most 64 threads' partial sums each within
(n / 64 + 16) 2^-24 of their value, taken here as 2^-20 for the sizes used; an
absolute error of 2^-20 in ln s, and one more rounding each of x - m, of the
product with ln 2 and of lse, give 2^-19 + 2^-22 |value| for log p and lse.
H weighs the same terms by up to ln n < 13: 13 2^-19.
"""
from __future__ import annotations

import math

import pytest
import torch

import software_pipelined_tiled_gemm_gb300 as sg

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    sg.check_operators()


def reference(logits, tokens, k):
    x = logits.double().cpu()
    lse = torch.logsumexp(x, 1)
    lp = x - lse[:, None]
    lp = torch.where(x == -INF, x, lp)
    p = lp.exp()
    h = -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(1)
    out = {"lse": lse, "entropy": h, "p": p, "lp": lp}
    if tokens is not None:
        t = tokens.cpu()
        out["logprobs"] = torch.where(t < 0, torch.zeros(len(t), dtype=torch.float64),
                                      lp.gather(1, t.clamp(min=0)[:, None])[:, 0])
    if k:
        ids = (x + 0.0).sort(dim=1, descending=True, stable=True).indices[:, :k]
        out["top_ids"], out["top_logprobs"] = ids, lp.gather(1, ids)
    return out


def close(got, want, name):
    got = got.double().cpu()
    fin = torch.isfinite(want)
    assert torch.equal(fin, torch.isfinite(got)), name
    assert torch.equal(got[~fin], want[~fin]) or torch.isnan(want[~fin]).any(), name
    tol = (13 if name == "entropy" else 1) * 2.0 ** -19 + 2.0 ** -22 * want[fin].abs()
    assert ((got[fin] - want[fin]).abs() <= tol).all(), (name, float((got[fin] - want[fin]).abs().max()))


def check(logits, tokens, k):
    r = sg.token_logprobs(logits, tokens, top_k=k)
    want = reference(logits, tokens, k)
    for name in ("lse", "entropy") + (("logprobs",) if tokens is not None else ()) + (("top_logprobs",) if k else ()):
        close(getattr(r, name), want[name], name)
    if k:
        assert torch.equal(r.top_ids.cpu(), want["top_ids"])
    return r, want


def logits_of(t, v, dt, seed, masked=False):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(t, v, generator=gen) * (0.5 + 3 * torch.rand(t, 1, generator=gen))
    if masked and v > 1:
        x[torch.rand(t, v, generator=gen) < 0.6] = -INF
        x[:, v // 2] = 1.0
    return x.to(DT[dt]).cuda(), torch.randint(0, v, (t,), generator=gen).cuda()


@pytest.mark.parametrize("t,v", [(1, 1), (1, 2), (1, 7), (3, 9), (1, 15), (2, 16), (1, 17), (5, 63), (1, 500), (2, 501),
                                 (17, 1000), (1, 4096), (1, 131072), (5, 131073), (300, 5003), (1, 70001),
                                 (1500, 2047), (800, 33001), (160, 65536)])
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_against_the_definition(t, v, dt):
    for masked in (False, True):
        x, tokens = logits_of(t, v, dt, seed=t + v, masked=masked)
        tokens[::5] = -100
        for k in (0, min(5, v)):
            check(x, tokens, k)


@pytest.mark.parametrize("k", [1, 2, 16, 17, 32, 33, 64])
def test_alternatives(k):
    for t, v, dt in ((3, 64, "f32"), (2, 100, "bf16"), (1, 131072, "bf16"), (900, 1003, "bf16"), (700, 20001, "f32"),
                     (20, 9001, "f16")):
        x, tokens = logits_of(t, v, dt, seed=k)
        check(x, tokens, k)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("t", [1, 500])
def test_ties_go_to_the_lowest_column(dt, t):
    v = 3001
    cols = torch.arange(v)
    for row in (torch.zeros(v), (cols % 3 == 1).float(), torch.where(cols % 2 == 0, -0.0, 0.0),
                (cols // 1000).float(), -(cols // 7).float().clamp(max=50), (cols >= v - 3).float()):
        x = row.to(DT[dt]).expand(t, v).contiguous().cuda()
        check(x, None, 64)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("t", [10, 1000])
def test_rows_with_nothing_or_almost_nothing_left(dt, t):
    v = 2600
    low = torch.finfo(DT[dt]).min
    x = torch.randn(t, v)
    x[0] = -INF
    x[1] = low
    x[2] = -INF
    x[2, 2100] = 3.0
    x[3] = low
    x[3, 11] = 0.5
    x[4] = -INF
    x[4, ::2] = low
    x[5] = torch.finfo(DT[dt]).max
    x[6] = 1000 + x[6]
    x[7] = -1000 - x[7].abs()
    x = x.to(DT[dt]).cuda()
    tokens = torch.full((t,), 11, device="cuda")
    r = sg.token_logprobs(x, tokens, top_k=6)
    for name, rows in (("logprobs", 0), ("lse", 0)):
        assert getattr(r, name)[rows] == -INF
    assert r.entropy[0] == 0 and r.top_ids[0].tolist() == [0, 1, 2, 3, 4, 5]
    assert (r.top_logprobs[0] == -INF).all()
    # a lowest value everywhere is a uniform row
    for row in (1, 5):
        assert abs(float(r.logprobs[row]) + math.log(v)) < 1e-5 and abs(float(r.entropy[row]) - math.log(v)) < 1e-4
        assert r.top_ids[row].tolist() == [0, 1, 2, 3, 4, 5]
    # one possible token: certain, exactly
    assert r.top_logprobs[2, 0] == 0 and r.entropy[2] == 0 and r.logprobs[2] == -INF
    assert r.top_ids[2].tolist() == [2100, 0, 1, 2, 3, 4]
    assert r.logprobs[3] == 0 and r.entropy[3] == 0 and r.top_ids[3, 0] == 11
    assert abs(float(r.top_logprobs[4, 0]) + math.log(v // 2)) < 1e-5
    check(x[6:].contiguous(), tokens[6:], 6)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("t", [2, 600])
def test_nan_and_infinity(dt, t):
    x, tokens = logits_of(t, 1500, dt, seed=1)
    clean = sg.token_logprobs(x, tokens, top_k=3)
    x[0, 40] = float("nan")
    x[1, 7] = INF
    x[1, 8] = -INF
    tokens[1] = 8
    r = sg.token_logprobs(x, tokens, top_k=3)
    assert math.isnan(r.lse[0]) and math.isnan(r.entropy[0]) and math.isnan(r.logprobs[0])
    assert r.top_ids[0, 0] == 40
    assert math.isnan(r.lse[1]) and math.isnan(r.entropy[1]) and r.logprobs[1] == -INF and r.top_ids[1, 0] == 7
    for a, b in zip(r, clean):
        assert torch.equal(a[2:], b[2:])


def test_largest_elements_in_one_threads_vectors():
    # More than the candidate list holds at or above the bound.
    for t in (1, 300):
        x = torch.randn(t, 200000)
        cols = torch.arange(200000)
        for stride in (128 * 4, 256 * 4):
            hot = (cols % stride) // 4 == 3
            y = torch.where(hot, 50 + (cols * 7919 % 1009).float() / 1009, x).cuda()
            got = sg.token_logprobs(y, None, top_k=64)
            want = y.cpu().sort(dim=1, descending=True, stable=True).indices[:, :64]
            assert torch.equal(got.top_ids.cpu(), want)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_rows_with_a_pitch_and_every_alignment(dt):
    t, v = 6, 1200
    x, tokens = logits_of(t, v, dt, seed=4)
    want, _ = check(x, tokens, 4)
    grad = torch.rand(t, device="cuda")
    dref = sg.token_logprobs_backward(x, tokens, want, grad, grad)
    for pitch, off in ((v, 0), (v + 1, 0), (v + 3, 1), (v + 8, 2), (v + 64, 5), (v, 7)):
        buf = torch.full((t * pitch + off,), float("nan"), dtype=x.dtype, device="cuda")
        view = buf[off:off + t * pitch].view(t, pitch)[:, :v]
        view.copy_(x)
        r = sg.token_logprobs(view, tokens, top_k=4)
        assert torch.equal(r.top_ids, want.top_ids)
        # the order of the sums follows the alignment, their value does not
        for a, b in zip(r[:4], want[:4]):
            assert torch.allclose(a, b, rtol=2 ** -21, atol=2 ** -18)
        d = sg.token_logprobs_backward(view, tokens, want, grad, grad)
        assert torch.equal(d, dref)
        into = torch.full_like(buf, 7.0)
        dview = into[off:off + t * pitch].view(t, pitch)[:, :v]
        sg.token_logprobs_backward(x, tokens, want, grad, grad, out=dview)
        assert torch.equal(dview, dref)
        dview.fill_(7.0)
        assert (into == 7.0).all()              # nothing beside the view was written


@pytest.mark.parametrize("t,v", [(1, 3), (4, 8), (7, 1001), (33, 4099), (300, 500), (2, 131072)])
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_gradient_against_the_formula(t, v, dt):
    for masked in (False, True):
        x, tokens = logits_of(t, v, dt, seed=t + v, masked=masked)
        tokens[::4] = -1
        r, want = check(x, tokens, 0)
        gen = torch.Generator().manual_seed(2)
        gl, gh = torch.randn(t, generator=gen), torch.randn(t, generator=gen)
        for a, b in ((gl, gh), (gl, None), (None, gh)):
            d = sg.token_logprobs_backward(x, tokens, r, None if a is None else a.cuda(),
                                           None if b is None else b.cuda()).double().cpu()
            p, lp = want["p"], want["lp"]
            counts = tokens.cpu() >= 0
            l64 = (torch.zeros(t) if a is None else a).double() * counts
            h64 = (torch.zeros(t) if b is None else b).double()
            plp = torch.where(p > 0, p * lp, torch.zeros_like(p))
            exact = -l64[:, None] * p - h64[:, None] * (plp + p * want["entropy"][:, None])
            exact[torch.arange(t), tokens.cpu().clamp(min=0)] += l64
            # p is within 2^-18 of its value (lse's rounding, 2^-19, and 2^t's), H as above
            tol = 2.0 ** -18 * (l64.abs()[:, None] * (p + (p > 0.5))
                                + h64.abs()[:, None] * (plp.abs() + p * (want["entropy"] + 13)[:, None])) + 1e-30
            u = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dt]
            tol = tol + u * (exact.abs() + tol) + (2.0 ** -24 if dt == "f16" else 1e-38)
            assert ((d - exact).abs() <= tol).all(), float(((d - exact).abs() / tol).max())


def test_gradient_against_differences():
    t, v = 5, 301
    x, tokens = logits_of(t, v, "f32", seed=9)
    r = sg.token_logprobs(x, tokens)
    gen = torch.Generator().manual_seed(10)
    gl, gh = torch.randn(t, generator=gen), torch.randn(t, generator=gen)
    d = sg.token_logprobs_backward(x, tokens, r, gl.cuda(), gh.cuda()).double().cpu()

    def value(z):
        lp = torch.log_softmax(z, 1)
        picked = lp.gather(1, tokens.cpu()[:, None])[:, 0]
        return (gl.double() * picked - gh.double() * (lp.exp() * lp).sum(1)).sum()

    z = x.double().cpu()
    for seed in range(4):
        w = torch.randn(t, v, generator=gen, dtype=torch.float64)
        step = 1e-4
        diff = (value(z + step * w) - value(z - step * w)) / (2 * step)
        # truncation step^2 / 6 times third derivatives of order 100; fp32 roundings 1e-5 of |d| |w|
        assert abs((d * w).sum() - diff) <= 1e-5 * (d.abs() * w.abs()).sum() + 1e-6


def test_gradient_in_place():
    x, tokens = logits_of(40, 2055, "bf16", seed=11)
    r = sg.token_logprobs(x, tokens)
    g = torch.rand(40, device="cuda")
    want = sg.token_logprobs_backward(x, tokens, r, g, g)
    got = sg.token_logprobs_backward(x, tokens, r, g, g, out=x)
    assert got is x and torch.equal(x, want)


def test_tokens_beyond_the_vocabulary_and_none():
    x, tokens = logits_of(4, 100, "f32", seed=12)
    tokens[1], tokens[2] = 100, -1
    r = sg.token_logprobs(x, tokens)
    assert math.isnan(r.logprobs[1]) and r.logprobs[2] == 0
    r = sg.token_logprobs(x, None, top_k=2)
    assert r.logprobs is None and r.top_ids.shape == (4, 2)
    r = sg.token_logprobs(x.view(2, 2, 100), tokens.view(2, 2), top_k=2)
    assert r.entropy.shape == (2, 2) and r.top_ids.shape == (2, 2, 2)
    empty = sg.token_logprobs(x[:0], tokens[:0], top_k=2)
    assert empty.logprobs.shape == (0,) and empty.top_ids.shape == (0, 2)
    assert sg.token_logprobs_backward(x[:0], tokens[:0], sg.token_logprobs(x[:0], tokens[:0])).shape == (0, 100)


def test_offsets_beyond_32_bits():
    t, v = 33000, 65536                      # 2.16e9 elements
    x = torch.zeros(t, v, dtype=torch.bfloat16, device="cuda")
    x[-1, 65000], x[32768, 3] = 8.0, 9.0
    tokens = torch.zeros(t, dtype=torch.int64, device="cuda")
    tokens[-1], tokens[32768] = 65000, 3
    r = sg.token_logprobs(x, tokens, top_k=1)
    assert r.top_ids[-1] == 65000 and r.top_ids[32768] == 3 and r.top_ids[5] == 0
    assert abs(float(r.logprobs[-1]) - (8 - math.log(65535 + math.exp(8)))) < 1e-5
    d = sg.token_logprobs_backward(x, tokens, r, torch.ones(t, device="cuda"), out=x)
    assert abs(float(d[-1, 65000]) - (1 - math.exp(float(r.logprobs[-1])))) < 2 ** -8
    assert abs(float(d[32768, 3]) - (1 - math.exp(float(r.logprobs[32768])))) < 2 ** -8


def test_rows_repeat_bit_for_bit():
    # Many rows per block, with the producer ahead of the search for alternatives.
    for t, v, k, dt in ((3000, 20000, 50, "f32"), (3000, 40000, 20, "bf16"), (2500, 9001, 64, "f16")):
        x, tokens = logits_of(64, v, dt, seed=k)
        x = x.repeat(t // 64 + 1, 1)[:t].contiguous()
        tokens = tokens.repeat(t // 64 + 1)[:t].contiguous()
        r = sg.token_logprobs(x, tokens, top_k=k)
        for field in r:
            lines = field[64:]
            period = field[:64].repeat(t // 64, *([1] * (field.dim() - 1)))[:t - 64]
            # odd row lengths shift the alignment, and with it the order of the sums
            if v % 8 == 0 or field.dtype == torch.int64:
                assert torch.equal(lines, period)
            else:
                assert torch.allclose(lines, period, rtol=2 ** -21, atol=2 ** -18)
        for _ in range(3):
            again = sg.token_logprobs(x, tokens, top_k=k)
            assert all(torch.equal(a, b) for a, b in zip(r, again))


def test_captured_in_a_graph():
    x, tokens = logits_of(50, 3000, "bf16", seed=20)
    g = torch.rand(50, device="cuda")
    side = torch.cuda.Stream()

    def run():
        r = sg.token_logprobs(x, tokens, top_k=5)
        return r + (sg.token_logprobs_backward(x, tokens, r, g, g),)
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = run()
    x.copy_(logits_of(50, 3000, "bf16", seed=21)[0])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, run()))


def test_refusals():
    x, tokens = logits_of(4, 50, "f32", seed=1)
    r = sg.token_logprobs(x, tokens)
    for bad in (dict(top_k=-1), dict(top_k=65), dict(top_k=51)):
        with pytest.raises(ValueError):
            sg.token_logprobs(x, tokens, **bad)
    with pytest.raises(TypeError):
        sg.token_logprobs(x.double(), tokens)
    with pytest.raises(TypeError):
        sg.token_logprobs(x, tokens.int())
    with pytest.raises(ValueError):
        sg.token_logprobs(x, tokens[:3])
    with pytest.raises(ValueError):
        sg.token_logprobs(x.t(), None)
    with pytest.raises(ValueError):
        sg.token_logprobs(x[:, :0], tokens)
    with pytest.raises(ValueError):
        sg.token_logprobs_backward(x, None, r, torch.ones(4, device="cuda"))
    with pytest.raises(ValueError):
        sg.token_logprobs_backward(x, tokens, r, torch.ones(5, device="cuda"))
    with pytest.raises(ValueError):
        sg.token_logprobs_backward(x, tokens, r, torch.ones(4, device="cuda").double())
    with pytest.raises(ValueError):
        sg.token_logprobs_backward(x, tokens, r, None, None, out=x.half())
    buf = torch.zeros(5, 50, device="cuda")
    with pytest.raises(sg.GemmError) as e:
        sg.token_logprobs_backward(buf[:4], tokens, r, None, None, out=buf[1:])
    assert e.value.status == sg.GEMM_ERR_INVALID_ARG and "overlaps" in str(e.value)
