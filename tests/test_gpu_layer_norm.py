"""Layer norm and its gradients on the GPU against the formulas in 64 bits.

Bounds.  u is half a step of the output's type relative to the value (2^-8
bf16, 2^-11 fp16, 2^-24 fp32).  A thread adds at most 32 columns of a row, or a
1024th of them, then come 5 steps between lanes and 32 between warps, so a
row's sum is off by at most c(n) = (max(32, n / 1024) + 48) 2^-23 times the sum
of absolute values; sums over rows likewise by their share of a block (152 or
more of them, or 8 rows), 8 warps and the blocks' partials.  rsqrt is within
2^-21 of its value.  The rest follows the formulas term by term.
"""
from __future__ import annotations

import pytest
import torch

import software_pipelined_tiled_gemm_gb300 as sg

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 1e-38, torch.float16: 2.0 ** -24, torch.float32: 1e-38}
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    sg.check_operators()


def c(n):
    return (max(32, n / 1024) + 48) * 2.0 ** -23


def c_rows(rows):
    return (rows / 152 + 8 + 48 + 16) * 2.0 ** -23


def rounded(value, bound, dtype):
    return value, bound + U[dtype] * (value.abs() + bound) + TINY[dtype]


def reference(x, w, b, dy, eps=EPS):
    """{name: (value, bound)}."""
    n = x.shape[1]
    wd = x.dtype if w is None else w.dtype
    x64, dy64 = x.double(), dy.double()
    w64 = torch.ones(n, dtype=torch.float64, device=x.device) if w is None else w.double()
    b64 = torch.zeros_like(w64) if b is None else b.double()
    mean = x64.mean(1, keepdim=True)
    d = x64 - mean
    rstd = 1 / (d.square().mean(1, keepdim=True) + eps).sqrt()
    h = d * rstd
    # The fp32 mean is off by c(n) |x| + 2^-24 |mean|; its lower part takes that out again.
    off = c(n) * x64.abs().mean(1, keepdim=True) + 2.0 ** -24 * mean.abs()
    spread = d.abs().mean(1, keepdim=True) + off
    e_r = c(n) * (1 + (off * rstd) ** 2) + 2.0 ** -21      # relative, of rstd
    e_h = rstd * (2.0 ** -23 * (d.abs() + off) + c(n) * spread) + h.abs() * e_r
    y = h * w64 + b64
    out = {"y": rounded(y, e_h * w64.abs() + 2.0 ** -23 * ((h * w64).abs() + b64.abs()), x.dtype)}
    g = dy64 * w64
    m1, m2 = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    e1 = (c(n) + 2.0 ** -23) * g.abs().mean(1, keepdim=True)
    e2 = (c(n) + 2.0 ** -22) * (g * h).abs().mean(1, keepdim=True) + (g.abs() * e_h).mean(1, keepdim=True)
    dx = rstd * (g - m1 - h * m2)
    e = rstd * (2.0 ** -22 * (g.abs() + m1.abs() + (h * m2).abs()) + e1 + (h.abs() + e_h) * e2 + m2.abs() * e_h)
    out["dx"] = rounded(dx, e * (1 + e_r) + dx.abs() * e_r, x.dtype)
    cr = c_rows(len(x))
    out["dweight"] = rounded((dy64 * h).sum(0), (dy64.abs() * e_h).sum(0) + cr * (dy64 * h).abs().sum(0), wd)
    out["dbias"] = rounded(dy64.sum(0), cr * dy64.abs().sum(0), wd)
    return out


def inputs(rows, cols, dt, wt, seed, bias=True):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")
    x = (normal(rows, cols) * 2 + normal(cols)).to(DT[dt])
    w = (1 + 0.2 * normal(cols)).to(DT[wt]) if wt else None
    b = normal(cols).to(DT[wt]) if wt and bias else None
    return x, w, b, normal(rows, cols).to(DT[dt])


def run_all(x, w, b, dy, eps=EPS):
    y, kept = sg.layer_norm(x, w, b, eps=eps, save=True)
    assert torch.equal(y, sg.layer_norm(x, w, b, eps=eps))
    return dict(zip(("y", "dx", "dweight", "dbias"), (y,) + sg.layer_norm_backward(dy, x, w, kept)))


def assert_within(got, want, what):
    value, bound = want
    assert got.shape == value.shape, what
    err = (got.double() - value).abs()
    assert bool((err <= bound).all()), (what, float((err / bound).max()))


COLS = [1, 2, 8, 31, 64, 257, 512, 520, 1000, 1024, 1025, 1531, 2048, 4096, 4097, 4104, 8192, 8200, 12000,
        16384, 16392, 20001, 28680, 32768, 32776, 40001]


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dt,wt", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"), ("f32", "f32")])
def test_output_and_gradients(cols, dt, wt):
    for rows in (1, 9, 333) if cols < 5000 else (3, 170):
        ts = inputs(rows, cols, dt, wt, seed=cols + rows)
        want = reference(*ts)
        for name, got in run_all(*ts).items():
            assert_within(got, want[name], (name, rows))


@pytest.mark.parametrize("rows,cols", [(5000, 64), (2047, 1531), (4100, 512)])
def test_many_rows(rows, cols):
    ts = inputs(rows, cols, "bf16", "f32", seed=1)
    want = reference(*ts)
    got, again = run_all(*ts), run_all(*ts)
    for name in got:
        assert_within(got[name], want[name], name)
        assert torch.equal(got[name], again[name]), name


@pytest.mark.parametrize("cols", [72, 1000, 6000, 33001])
def test_without_weight_or_bias(cols):
    x, w, b, dy = inputs(20, cols, "f16", None, seed=2)
    want = reference(x, None, None, dy)
    for name, got in run_all(x, None, None, dy).items():
        assert_within(got, want[name], name)
    x, w, b, dy = inputs(20, cols, "f16", "f16", seed=3)
    assert_within(sg.layer_norm(x, w), reference(x, w, None, dy)["y"], "no bias")
    assert_within(sg.layer_norm(x, None, b), reference(x, None, b, dy)["y"], "no weight")


@pytest.mark.parametrize("cols", [48, 700, 5000, 33000])
def test_rows_far_from_zero_keep_their_differences(cols):
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(12, cols, generator=gen, device="cuda") + 10.0 ** torch.arange(-1.0, 5.0, 0.5, device="cuda")[:, None]
    dy = torch.randn(12, cols, generator=gen, device="cuda")
    w = torch.randn(cols, generator=gen, device="cuda")
    want = reference(x, w, None, dy)
    for name, got in run_all(x, w, None, dy).items():
        assert_within(got, want[name], name)


@pytest.mark.parametrize("cols", [40, 1000, 9000, 33000])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_large_and_small_values(cols, dt):
    """Squares beyond fp32's range, and variances below eps."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    for size in (1e30, 1e18, 1e-12, 1e-25):
        x = (torch.randn(6, cols, generator=gen, device="cuda") * size).to(DT[dt])
        dy = torch.randn(6, cols, generator=gen, device="cuda").to(DT[dt])
        want = reference(x, None, None, dy)
        y, kept = sg.layer_norm(x, save=True)
        dx = sg.layer_norm_backward(dy, x, None, kept, need=(True, False, False))[0]
        assert_within(y, want["y"], ("y", size))
        value, bound = want["dx"]
        assert_within(dx, (value, bound + 1e-37), ("dx", size))   # (subnormal factors of 1e-30)


@pytest.mark.parametrize("cols", [5, 300, 3000, 33000])
def test_constant_rows_and_rows_with_nan_or_infinity(cols):
    x = torch.full((6, cols), 3.25, device="cuda").bfloat16()
    x[1, cols // 2], x[3, 0], x[4, -1] = float("nan"), float("inf"), float("-inf")
    b = torch.arange(cols, device="cuda").bfloat16()
    y = sg.layer_norm(x, None, b)
    # The mean's rounding leaves a constant row differences, which the second sum takes out but
    # for its own rounding: rstd c(n) off, as in the other rows.
    constant = [0, 2, 5]
    assert_within(y[constant], reference(x[constant], None, b, x[constant])["y"], "constant")
    for r in (1, 3, 4):
        assert y[r].isnan().all()


@pytest.mark.parametrize("cols", [24, 1536, 1531, 12000, 33000])
def test_pitch_alignment_and_in_place(cols):
    x, w, b, dy = inputs(37, cols, "bf16", "bf16", seed=6)
    want = reference(x, w, b, dy)
    same = run_all(x, w, b, dy)
    for shift in (0, 1, 8):
        def wide(t):
            big = torch.full((len(t), cols + 16), float("nan"), dtype=t.dtype, device="cuda")
            big[:, shift:shift + cols] = t
            return big[:, shift:shift + cols]

        def odd(t):
            flat = torch.full((t.numel() + 16,), float("nan"), dtype=t.dtype, device="cuda")
            flat[shift:shift + t.numel()] = t.reshape(-1)
            return flat[shift:shift + t.numel()].view(t.shape)
        for name, got in run_all(wide(x), odd(w), odd(b), wide(dy)).items():
            assert_within(got, want[name], (name, shift))
        outs = odd(x), odd(w), odd(w)
        y, kept = sg.layer_norm(x, w, b, out=outs[0], save=True)
        assert y is outs[0]
        assert_within(y, want["y"], ("y", shift))
        got = sg.layer_norm_backward(dy, x, w, kept, out=outs)
        assert got[0] is outs[0]
        for name, t in zip(("dx", "dweight", "dbias"), got):
            assert_within(t, want[name], (name, shift))
    y, kept = sg.layer_norm(x, w, b, save=True)
    d = dy.clone()
    assert torch.equal(sg.layer_norm_backward(d, x, w, kept, out=(d, None, None))[0], same["dx"])
    z = x.clone()
    assert torch.equal(sg.layer_norm(z, w, b, out=z), same["y"])


@pytest.mark.parametrize("cols", [1, 3, 13, 61, 1019, 1531, 4099])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_share_vectors_of_memory_and_nothing_else(cols, dt):
    """A row that begins or ends inside 16 bytes has neighbours there: rows of NaN
    between clean ones, in every place of a vector, out of place and in place."""
    x, w, b, dy = inputs(67, cols, dt, "f32", seed=12)
    want = reference(x, w, b, dy)
    clean = torch.arange(67, device="cuda") % 2 == 0
    for at in (0, 1, 3):
        def placed(t):
            flat = torch.full((t.numel() + 16,), float("nan"), dtype=t.dtype, device="cuda")
            out = flat[at:at + t.numel()].view(t.shape)
            out.copy_(t)
            out[~clean] = float("nan")
            return flat, out
        (_, px), (flat_d, pd) = placed(x), placed(dy)
        y, kept = sg.layer_norm(px, w, b, save=True)
        dx = sg.layer_norm_backward(pd, px, w, kept, need=(True, False, False))[0]
        flat_x, z = placed(x)
        sg.layer_norm(z, w, b, out=z)
        sg.layer_norm_backward(pd, px, w, kept, need=(True, False, False), out=(pd, None, None))
        for name, got in (("y", y), ("dx", dx), ("y", z), ("dx", pd)):
            value, bound = want[name]
            assert_within(got[clean], (value[clean], bound[clean]), (name, at))
            assert got[~clean].isnan().all()
        for flat in (flat_x, flat_d):   # beside the matrix nothing is written
            assert flat[:at].isnan().all() and flat[at + x.numel():].isnan().all()


def test_each_gradient_alone_and_no_rows():
    x, w, b, dy = inputs(50, 264, "f32", "f32", seed=7)
    y, kept = sg.layer_norm(x, w, b, save=True)
    full = sg.layer_norm_backward(dy, x, w, kept)
    for i in range(3):
        need = tuple(j == i for j in range(3))
        got = sg.layer_norm_backward(dy, x, w, kept, need=need)
        assert torch.equal(got[i], full[i]) and sum(t is None for t in got) == 2
    assert sg.layer_norm_backward(dy, x, w, kept, need=(False,) * 3) == (None, None, None)
    y, kept = sg.layer_norm(x[:0], w, b, save=True)
    dx, dw, db = sg.layer_norm_backward(dy[:0], x[:0], w, kept)
    assert y.shape == dx.shape == (0, 264) and not dw.any() and not db.any()


def test_leading_dimensions():
    x, w, b, dy = inputs(24, 136, "bf16", "bf16", seed=8)
    want = run_all(x, w, b, dy)
    got = run_all(x.view(2, 3, 4, 136), w, b, dy.view(2, 3, 4, 136))
    for name in want:
        assert torch.equal(got[name].reshape(want[name].shape), want[name])
    one = sg.layer_norm(x[3], w, b)
    assert one.shape == (136,) and torch.equal(one, want["y"][3])


def test_against_differences():
    """<dy, y(x + t v) - y(x - t v)> / 2t against <dx, v>, in fp32."""
    x, w, b, dy = inputs(16, 640, "f32", "f32", seed=9)
    v = torch.randn(x.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    t = 2.0 ** -7
    got = run_all(x, w, b, dy)
    diff = (dy.double() * (sg.layer_norm(x + t * v, w, b).double() - sg.layer_norm(x - t * v, w, b).double())).sum() / (2 * t)
    # Rounding of the outputs over 2t, and the third derivative's t^2 part: below t^2 of the sizes.
    scale = dy.double().norm() * v.double().norm()
    assert abs(diff - (got["dx"].double() * v.double()).sum()) <= (2.0 ** -22 / t + t * t) * scale


def test_streams_and_graph():
    x, w, b, dy = inputs(300, 1032, "bf16", "f32", seed=10)
    want = run_all(x, w, b, dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run_all(x, w, b, dy)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, kept = sg.layer_norm(x, w, b, save=True)
        held = (y,) + sg.layer_norm_backward(dy, x, w, kept)
    new = inputs(300, 1032, "bf16", "f32", seed=11)
    expect = run_all(*new)
    for name in want:
        assert torch.equal(got[name], want[name]), name
    for a, t in zip((x, w, b, dy), new):
        a.copy_(t)
    graph.replay()
    torch.cuda.synchronize()
    for name, t in zip(("y", "dx", "dweight", "dbias"), held):
        assert torch.equal(t, expect[name]), name
