"""The gated feed-forward block on the GPU against its formulas in 64 bits.

Bounds.  With u the unit roundoff of the 16-bit type (2^-8 bf16, 2^-11 fp16)
and c(K) = (K + 16) 2^-23 for a K-term fp32 sum, whatever its order, each
quantity's error is bounded element by element from the roundings the
operator makes (H, dG and dU to the type, every sum in fp32, the output once)
through the absolute values of what it multiplies.  The activations' fp32
evaluation is within 2^-19 of their values.
"""
from __future__ import annotations

import pytest
import torch

import software_pipelined_tiled_gemm_gb300 as sg

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"bf16": 1e-38, "f16": 2.0 ** -24}   # half the spacing below the normal range, twice over


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    sg.check_operators()


def c(k):
    return (k + 16) * 2.0 ** -23


def act64(name, g):
    """The activation, its derivative, and a bound of its second derivative."""
    if name == "relu":
        return g.clamp(min=0), (g > 0).double(), 0.0
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s)), 0.5
    k = 0.7978845608
    t = torch.tanh(k * (g + 0.044715 * g ** 3))
    return (0.5 * g * (1 + t),
            0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g), 1.2)


def inputs(m, d, i, dt, seed):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(m, d, generator=gen).to(DT[dt])
    w_in = (torch.randn(2 * i, d, generator=gen) * d ** -0.5).to(DT[dt])
    w_out = (torch.randn(d, i, generator=gen) * i ** -0.5).to(DT[dt])
    dy = torch.randn(m, d, generator=gen).to(DT[dt])
    return x, w_in, w_out, dy


def reference(x, w_in, w_out, dy, act, dt):
    """{name: (value, bound)} of the output and the gradients."""
    u, eps = U[dt], 2.0 ** -19
    x, w_in, w_out, dy = (t.double() for t in (x, w_in, w_out, dy))
    m, d = x.shape
    i = w_out.shape[1]
    gu, e_gu = x @ w_in.T, c(d) * (x.abs() @ w_in.abs().T)
    g, up, e_g, e_u = gu[:, :i], gu[:, i:], e_gu[:, :i], e_gu[:, i:]
    a, da, curve = act64(act, g)
    h = a * up
    e_a = da.abs() * e_g + curve * e_g ** 2 + eps * a.abs()
    e_h = e_a * up.abs() + (a.abs() + e_a) * e_u + 2 * u * h.abs() + TINY[dt]
    out = {"y": (h @ w_out.T, (e_h + c(i) * h.abs()) @ w_out.abs().T)}
    dh, e_dh = dy @ w_out, c(d) * (dy.abs() @ w_out.abs())
    # The derivative moves by curve e_g; ReLU's jumps where g may be on either side of 0.
    e_da = curve * e_g + eps * (da.abs() + 1e-3)
    if act == "relu":
        e_da = e_da + (g.abs() <= e_g).double()
    dg, du = dh * up * da, dh * a
    e_dg = (e_dh * (up * da).abs() + dh.abs() * e_u * da.abs() + (dh * up).abs() * e_da) * 1.01 \
        + 2 * u * dg.abs() + TINY[dt]
    e_du = (e_dh * a.abs() + dh.abs() * e_a) * 1.01 + 2 * u * du.abs() + TINY[dt]
    dgu, e_dgu = torch.cat([dg, du], 1), torch.cat([e_dg, e_du], 1)
    out["dx"] = (dgu @ w_in, (e_dgu + c(2 * i) * dgu.abs()) @ w_in.abs())
    out["dw_in"] = (dgu.T @ x, (e_dgu + c(m) * dgu.abs()).T @ x.abs())
    out["dw_out"] = (dy.T @ h, dy.abs().T @ (e_h + c(m) * h.abs()))
    return {k: (v, b + u * (v.abs() + b) + TINY[dt]) for k, (v, b) in out.items()}


def assert_within(got, want, what):
    value, bound = want
    err = (got.double().cpu() - value).abs()
    worst = (err / bound).max().item() if err.numel() else 0.0
    assert not err.numel() or worst <= 1.0, (what, worst)


def run_all(x, w_in, w_out, dy, act):
    y, kept = sg.gated_ffn(x, w_in, w_out, act=act, save=True)
    grads = sg.gated_ffn_backward(dy, x, w_in, w_out, kept)
    return dict(zip(("y", "dx", "dw_in", "dw_out"), (y,) + grads))


SIZES = [
    (1, 64, 64), (1, 2048, 1024), (2, 72, 8), (5, 128, 192), (17, 1, 1), (33, 67, 101), (64, 512, 640),
    (65, 640, 512), (100, 96, 264), (128, 256, 128), (129, 255, 257), (257, 1531, 129), (300, 512, 1408),
    (515, 520, 72), (640, 512, 1408), (1000, 136, 2050), (1030, 1024, 1032),
]


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("act,dt", [("silu", "bf16"), ("gelu", "f16"), ("relu", "bf16")])
def test_output_and_gradients(size, act, dt):
    ts = inputs(*size, dt, seed=sum(size))
    want = reference(*ts, act, dt)
    got = run_all(*(t.cuda() for t in ts), act)
    for name in want:
        assert_within(got[name], want[name], (name, size))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_gradients_against_differences(dt):
    # <grad, v> against central differences of <dy, y> along v, both sides of
    # the difference in 64 bits: truncation h^2 / 6 times a third derivative
    # of order 10 here, next to the gradients' own bound.
    m, d, i = 40, 48, 56
    x, w_in, w_out, dy = inputs(m, d, i, dt, seed=3)
    got = run_all(x.cuda(), w_in.cuda(), w_out.cuda(), dy.cuda(), "silu")
    want = reference(x, w_in, w_out, dy, "silu", dt)
    point = [t.double() for t in (x, w_in, w_out)]

    def value(p):
        gu = p[0] @ p[1].T
        return ((act64("silu", gu[:, :i])[0] * gu[:, i:]) @ p[2].T * dy.double()).sum()

    gen = torch.Generator().manual_seed(4)
    for k, name in enumerate(("dx", "dw_in", "dw_out")):
        v = torch.randn(point[k].shape, generator=gen, dtype=torch.float64)
        step = 1e-5
        hi, lo = list(point), list(point)
        hi[k] = point[k] + step * v
        lo[k] = point[k] - step * v
        diff = (value(hi) - value(lo)) / (2 * step)
        mine = (got[name].double().cpu() * v).sum()
        bound = (want[name][1] * v.abs()).sum() + 1e-4
        assert abs(mine - diff) <= bound, (name, float(mine), float(diff), float(bound))


def test_rows_with_a_pitch_and_unaligned_bases():
    m, d, i = 70, 200, 96
    x, w_in, w_out, dy = inputs(m, d, i, "bf16", seed=8)
    want = reference(x, w_in, w_out, dy, "silu", "bf16")
    for pitch, off in ((d + 24, 8), (d + 3, 1)):
        def place(t):
            buf = torch.full((m * pitch + off + 8,), float("nan"), dtype=t.dtype, device="cuda")
            view = buf[off:off + m * pitch].view(m, pitch)[:, :d]
            view.copy_(t)
            return view
        got = run_all(place(x), w_in.cuda(), w_out.cuda(), place(dy), "silu")
        for name in want:
            assert_within(got[name], want[name], (name, pitch, off))


def test_weights_at_an_odd_address():
    m, d, i = 20, 64, 48
    x, w_in, w_out, dy = inputs(m, d, i, "f16", seed=9)

    def odd(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        view = buf[1:].view(t.shape)
        view.copy_(t)
        return view
    got = run_all(x.cuda(), odd(w_in), odd(w_out), dy.cuda(), "gelu")
    want = reference(x, w_in, w_out, dy, "gelu", "f16")
    for name in want:
        assert_within(got[name], want[name], name)


@pytest.mark.parametrize("size", [(33, 67, 101), (130, 256, 72), (1, 40, 24)], ids=str)
def test_nothing_is_written_outside_the_outputs(size):
    x, w_in, w_out, dy = (t.cuda() for t in inputs(*size, "bf16", seed=5))
    m, d, i = size
    y0, kept = sg.gated_ffn(x, w_in, w_out, save=True)
    g0 = sg.gated_ffn_backward(dy, x, w_in, w_out, kept)

    def framed(shape):
        n = shape[0] * shape[1]
        buf = torch.full((n + 128,), 7.0, dtype=torch.bfloat16, device="cuda")
        return buf, buf[64:64 + n].view(shape)
    frames = [framed(s) for s in ((m, d), (m, d), (2 * i, d), (d, i))]
    sg.gated_ffn(x, w_in, w_out, out=frames[0][1])
    sg.gated_ffn_backward(dy, x, w_in, w_out, kept, out=tuple(f[1] for f in frames[1:]))
    for (buf, view), want in zip(frames, (y0,) + g0):
        assert torch.equal(view, want)
        assert (buf[:64] == 7).all() and (buf[64 + view.numel():] == 7).all()


def test_no_tokens():
    _, w_in, w_out, _ = (t.cuda() for t in inputs(1, 32, 48, "bf16", seed=1))
    x = torch.empty(0, 32, dtype=torch.bfloat16, device="cuda")
    y, kept = sg.gated_ffn(x, w_in, w_out, save=True)
    assert y.shape == (0, 32)
    dx, dw_in, dw_out = sg.gated_ffn_backward(x, x, w_in, w_out, kept)
    assert dx.shape == (0, 32) and not dw_in.any() and not dw_out.any()


def test_leading_dimensions_needed_gradients_and_given_outputs():
    x, w_in, w_out, dy = (t.cuda() for t in inputs(24, 64, 40, "f16", seed=2))
    flat, kept = sg.gated_ffn(x, w_in, w_out, save=True)
    y, kept3 = sg.gated_ffn(x.view(2, 3, 4, 64), w_in, w_out, save=True)
    assert y.shape == (2, 3, 4, 64) and torch.equal(y.view(24, 64), flat)
    all3 = sg.gated_ffn_backward(dy, x, w_in, w_out, kept)
    for k in range(3):
        need = tuple(j == k for j in range(3))
        one = sg.gated_ffn_backward(dy, x, w_in, w_out, kept, need=need)
        assert [t is not None for t in one] == list(need) and torch.equal(one[k], all3[k])
    dx = sg.gated_ffn_backward(dy.view(2, 3, 4, 64), x.view(2, 3, 4, 64), w_in, w_out, kept3)[0]
    assert torch.equal(dx.view(24, 64), all3[0])


def test_repeats_bit_for_bit_and_on_two_streams():
    ts = [t.cuda() for t in inputs(200, 512, 704, "bf16", seed=6)]
    first = run_all(*ts, "silu")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    results = []
    for rep in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                results.append(run_all(*ts, "silu"))
    torch.cuda.synchronize()
    for r in results:
        for name in first:
            assert torch.equal(r[name], first[name]), name


def test_captured_in_a_graph():
    x, w_in, w_out, dy = (t.cuda() for t in inputs(96, 256, 320, "bf16", seed=7))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run_all(x, w_in, w_out, dy, "silu")       # the stream's handle exists before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = run_all(x, w_in, w_out, dy, "silu")
    for seed in (11, 12):
        for t, new in zip((x, w_in, w_out, dy), inputs(96, 256, 320, "bf16", seed=seed)):
            t.copy_(new)
        graph.replay()
        want = run_all(x, w_in, w_out, dy, "silu")
        torch.cuda.synchronize()
        for name in want:
            assert torch.equal(got[name], want[name]), name


def test_infinities_and_nan_stay_in_their_rows():
    x, w_in, w_out, _ = (t.cuda() for t in inputs(40, 64, 48, "bf16", seed=13))
    clean = sg.gated_ffn(x, w_in, w_out)
    x[3, 5], x[37, 0] = float("nan"), float("inf")
    y = sg.gated_ffn(x, w_in, w_out)
    bad = torch.zeros(40, dtype=torch.bool)
    bad[[3, 37]] = True
    assert not torch.isfinite(y[bad]).any()
    assert torch.equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
def test_large_gates_saturate(act):
    # Gates of +-1000: act(g) is g or 0 and its derivative 1 or 0, never NaN.
    m, d, i = 8, 8, 8
    x = torch.eye(8, dtype=torch.bfloat16).cuda()
    w_in = torch.cat([torch.full((i, d), -1000.0), torch.ones(i, d)]).to(torch.bfloat16).cuda()
    w_in[:4] = 1000.0
    w_out = torch.eye(8, dtype=torch.bfloat16).cuda()
    y, kept = sg.gated_ffn(x, w_in, w_out, act=act, save=True)
    assert torch.equal(y.float(), torch.tensor([1000.0] * 4 + [0.0] * 4).cuda().expand(8, 8))
    dx, dw_in, dw_out = sg.gated_ffn_backward(torch.ones_like(y), x, w_in, w_out, kept)
    assert torch.isfinite(dx).all() and torch.isfinite(dw_in).all() and torch.isfinite(dw_out).all()
    assert torch.equal(dw_in[:8].float(), torch.tensor([1.0] * 4 + [0.0] * 4).cuda()[:, None].expand(8, 8))


def test_refusals():
    x, w_in, w_out, dy = (t.cuda() for t in inputs(8, 32, 16, "bf16", seed=1))
    _, kept = sg.gated_ffn(x, w_in, w_out, save=True)
    with pytest.raises(TypeError):
        sg.gated_ffn(x.float(), w_in.float(), w_out.float())
    with pytest.raises(TypeError):
        sg.gated_ffn(x, w_in.half(), w_out)
    with pytest.raises(ValueError):
        sg.gated_ffn(x, w_in[:-1], w_out)
    with pytest.raises(ValueError):
        sg.gated_ffn(x[:, :-1], w_in, w_out)
    with pytest.raises(ValueError):
        sg.gated_ffn(x, w_in.t().contiguous().t(), w_out)
    with pytest.raises(ValueError):
        sg.gated_ffn(x.t().contiguous().t(), w_in, w_out)
    with pytest.raises(ValueError):
        sg.gated_ffn(x, w_in, w_out, out=torch.empty(8, 31, dtype=x.dtype, device="cuda"))
    with pytest.raises(ValueError):
        sg.gated_ffn(x, w_in.cpu(), w_out)
    with pytest.raises(ValueError):
        sg.gated_ffn_backward(dy[:-1], x, w_in, w_out, kept)
    with pytest.raises(ValueError):
        sg.gated_ffn_backward(dy[:4], x[:4], w_in, w_out, kept)
    with pytest.raises(sg.GemmError) as e:
        sg.gated_ffn(x, w_in, w_out, out=x)
    assert e.value.status == sg.GEMM_ERR_INVALID_ARG and "overlaps" in str(e.value)
    with pytest.raises(sg.GemmError):
        sg.gated_ffn_backward(dy, x, w_in, w_out, kept, out=(None, w_in, None))


# A few tokens take another path (passes over the weights), product by product
# where their values fit on chip: token counts around its steps, widths around
# its groups of 8 and 16 rows and 32 elements of K, and both mixed cases.
FEW = [(1, 32, 8), (2, 33, 7), (3, 1, 300), (4, 255, 1), (7, 1000, 513), (8, 64, 2440), (9, 520, 1217), (15, 96, 1224),
       (16, 1031, 136), (24, 160, 2433), (31, 72, 264), (32, 2050, 40), (33, 72, 264)]


@pytest.mark.parametrize("size", FEW, ids=str)
@pytest.mark.parametrize("act,dt", [("silu", "bf16"), ("gelu", "f16")])
def test_few_tokens(size, act, dt):
    ts = inputs(*size, dt, seed=sum(size))
    want = reference(*ts, act, dt)
    for k, v in run_all(*(t.cuda() for t in ts), act).items():
        assert_within(v, want[k], (size, k))


@pytest.mark.parametrize("size", [(1, 200, 40000), (6, 17000, 24), (7, 24, 17000), (32, 64, 3300), (32, 8200, 64),
                                  (1, 120000, 8)], ids=str)
def test_few_tokens_with_long_rows(size):
    x, w_in, w_out, _ = inputs(*size, "bf16", seed=sum(size))
    want = reference(x, w_in, w_out, torch.zeros_like(x), "relu", "bf16")["y"]
    assert_within(sg.gated_ffn(x.cuda(), w_in.cuda(), w_out.cuda(), act="relu"), want, size)


def test_few_tokens_do_not_meet():
    x, w_in, w_out, _ = inputs(6, 100, 60, "bf16", seed=3)
    xs, w_in, w_out = x.cuda(), w_in.cuda(), w_out.cuda()
    ref = sg.gated_ffn(xs, w_in, w_out)
    for bad in (float("inf"), float("nan")):
        spoilt = xs.clone()
        spoilt[2, 99] = bad
        got = sg.gated_ffn(spoilt, w_in, w_out)
        keep = [0, 1, 3, 4, 5]
        assert torch.equal(got[keep], ref[keep]) and not torch.isfinite(got[2]).all()
    buf = torch.full((6, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    buf[:, :100] = xs
    assert torch.equal(sg.gated_ffn(buf[:, :100], w_in, w_out), ref)


def test_few_tokens_follow_an_update_of_the_weights():
    """The weights are read as the kernels before the call on the stream left them."""
    x, w_in, w_out, _ = (t.cuda() for t in inputs(2, 2048, 4096, "bf16", seed=4))
    w2, o2 = torch.zeros_like(w_in), torch.zeros_like(w_out)
    want = sg.gated_ffn(x, w_in, w_out)
    for _ in range(20):
        w2.zero_()
        o2.zero_()
        sg.gated_ffn(x, w2, o2)
        w2.copy_(w_in)
        o2.copy_(w_out)
        assert torch.equal(sg.gated_ffn(x, w2, o2), want)


@pytest.mark.parametrize("offsets", [(1, 3, 5), (0, 1, 0), (8, 8, 7)], ids=str)
@pytest.mark.parametrize("size", [(1, 64, 48), (6, 129, 77), (20, 40, 23)], ids=str)
def test_few_tokens_read_operands_where_they_lie(size, offsets):
    m, d, i = size
    x, w_in, w_out, _ = (t.cuda() for t in inputs(m, d, i, "bf16", seed=5))
    ref = sg.gated_ffn(x, w_in, w_out)

    def moved(t, k):
        buf = torch.full((t.numel() + 32,), float("nan"), dtype=t.dtype, device="cuda")
        out = buf[k:k + t.numel()].view(t.shape)
        return out.copy_(t)
    ts = [moved(t, k) for t, k in zip((x, w_in, w_out), offsets)]
    assert torch.equal(sg.gated_ffn(*ts), ref)
    rows = torch.full((m, d + 5), float("nan"), dtype=x.dtype, device="cuda")
    rows[:, 2:2 + d] = x
    assert torch.equal(sg.gated_ffn(rows[:, 2:2 + d], w_in, w_out), ref)
