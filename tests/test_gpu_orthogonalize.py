"""The orthogonalised update on the GPU against its iteration in 64 bits.

The iteration amplifies errors along small singular values, so no bound by
element holds for it.  The tolerance is the distance of a model from the
exact result: the same iteration in 64 bits with its iterates rounded to fp16
where the kernels round them (X 2^8, A and B), and the result to bf16.  The
kernels' other errors, fp32 sums, are 2^-12 of those roundings; a factor of
1.5 covers how far the random parts of two such errors differ.
"""
from __future__ import annotations

import pytest
import torch

import software_pipelined_tiled_gemm_gb300 as sg

pytestmark = pytest.mark.gpu

COEFFS = (3.4445, -4.7750, 2.0315)
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    sg.check_operators()


def iterate(g, steps=5, coeffs=COEFFS, eps=1e-7, rounded=False):
    g = g.double()
    s = 256.0
    q = (lambda t: t.half().double()) if rounded else (lambda t: t)
    x = q(g * (s / g.norm().clamp(min=eps)))
    a, b, c = coeffs
    tall = x.shape[0] > x.shape[1]
    for k in range(steps):
        p = q((x.T @ x if tall else x @ x.T) / (s * s))
        w = q(b * p + c * (p @ p))
        x = a * x + (x @ w if tall else w @ x)
        if k + 1 < steps:
            x = q(x)
    x = x / s
    return x.bfloat16().double() if rounded else x


def gradient(m, n, seed, scale=1e-3):
    gen = torch.Generator().manual_seed(seed)
    r = max(1, min(m, n) // 16)
    return (torch.randn(m, r, generator=gen) @ torch.randn(r, n, generator=gen) * 2 / r ** 0.5
            + torch.randn(m, n, generator=gen)) * scale


def check(got, g, **kw):
    exact, model = iterate(g, **kw), iterate(g, rounded=True, **kw)
    scale = exact.norm()
    off = float((got.double().cpu() - exact).norm() / scale)
    tol = 1.5 * float((model - exact).norm() / scale) + 2.0 ** -9
    assert off <= tol, (tuple(g.shape), off, tol)


@pytest.mark.parametrize("shape", [(1, 1), (1, 77), (33, 1), (8, 8), (64, 64), (100, 200), (200, 100), (127, 129),
                                   (256, 640), (257, 513), (640, 256), (500, 499), (1000, 300), (300, 1032),
                                   (2049, 96), (70, 3000), (513, 1100)], ids=str)
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_against_the_iteration(shape, dt):
    g = gradient(*shape, seed=shape[0] + shape[1]).to(DT[dt])
    check(sg.orthogonalize(g.cuda()), g)


def test_scale_of_the_gradient_does_not_matter():
    g = gradient(96, 160, seed=1)
    ref = sg.orthogonalize(g.cuda())
    for k in (-60, -20, 20, 40):
        # a power of two changes no rounding but that of the norm's fp32 value
        got = sg.orthogonalize((g * 2.0 ** k).cuda(), eps=1e-30)
        assert (got.double() - ref.double()).norm() <= 2.0 ** -9 * ref.double().norm(), k


def test_singular_values_end_near_one():
    s = torch.linalg.svdvals(sg.orthogonalize(gradient(128, 256, seed=2).cuda()).double().cpu())
    assert s.max() < 1.25 and s.min() > 0.6


def test_transposed_input_gives_the_transpose():
    g = gradient(120, 200, seed=3)
    a, b = sg.orthogonalize(g.cuda()), sg.orthogonalize(g.T.contiguous().cuda())
    assert (a.double() - b.T.double()).norm() <= 6e-3 * a.double().norm()


@pytest.mark.parametrize("b,m,n", [(3, 64, 64), (8, 100, 264), (5, 257, 65), (2, 640, 512)])
def test_batch_is_its_matrices(b, m, n):
    g = torch.stack([gradient(m, n, seed=10 + i, scale=10.0 ** -i) for i in range(b)])
    got = sg.orthogonalize(g.cuda())
    for i in range(b):
        check(got[i], g[i])


def test_rows_with_a_pitch_and_odd_addresses():
    m, n = 60, 72
    g = gradient(m, n, seed=4)
    for dt in (torch.float32, torch.bfloat16):
        ref = sg.orthogonalize(g.to(dt).cuda())
        for pitch, off in ((n + 8, 0), (n + 5, 3)):
            buf = torch.full((m * pitch + off,), float("nan"), dtype=dt, device="cuda")
            view = buf[off:].view(m, pitch)[:, :n]
            view.copy_(g)
            assert torch.equal(sg.orthogonalize(view), ref)
    batch = torch.stack([g, g * 2, g * 3]).cuda()
    assert torch.equal(sg.orthogonalize(batch[::2]), sg.orthogonalize(batch[::2].contiguous()))


@pytest.mark.parametrize("steps", [1, 2, 7])
def test_steps_and_coefficients(steps):
    g = gradient(80, 96, seed=5)
    cubic = (1.5, -0.5, 0.0)
    check(sg.orthogonalize(g.cuda(), steps=steps), g, steps=steps)
    check(sg.orthogonalize(g.cuda(), steps=steps, coeffs=cubic), g, steps=steps, coeffs=cubic)


def test_zero_and_tiny_matrices():
    assert not sg.orthogonalize(torch.zeros(40, 56, device="cuda")).any()
    tiny = torch.full((16, 16), 1e-30, device="cuda")   # below eps: scaled by 1 / eps, stays tiny
    assert sg.orthogonalize(tiny).abs().max() < 1e-10


def test_empty_and_nothing_outside_the_output():
    for shape in ((0, 5), (5, 0), (0, 4, 4)):
        assert sg.orthogonalize(torch.zeros(shape, device="cuda")).shape == shape
    g = gradient(33, 51, seed=6).cuda()
    buf = torch.full((33 * 51 + 100,), 9.0, dtype=torch.bfloat16, device="cuda")
    out = buf[50:50 + 33 * 51].view(33, 51)
    sg.orthogonalize(g, out=out)
    assert torch.equal(out, sg.orthogonalize(g))
    assert (buf[:50] == 9).all() and (buf[50 + 33 * 51:] == 9).all()


def test_nan_in_one_matrix_leaves_the_others():
    g = torch.stack([gradient(48, 64, seed=i) for i in range(3)]).cuda()
    clean = sg.orthogonalize(g)
    g[1, 7, 9] = float("nan")
    got = sg.orthogonalize(g)
    assert torch.isnan(got[1]).any()
    assert torch.equal(got[0], clean[0]) and torch.equal(got[2], clean[2])


def test_repeats_bit_for_bit_and_in_a_graph():
    g = gradient(300, 420, seed=7).cuda()
    ref = sg.orthogonalize(g)
    for _ in range(3):
        assert torch.equal(sg.orthogonalize(g), ref)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        sg.orthogonalize(g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = sg.orthogonalize(g)
    g.copy_(gradient(300, 420, seed=8))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, sg.orthogonalize(g))


def test_refusals():
    g = torch.zeros(8, 8, device="cuda")
    with pytest.raises(TypeError):
        sg.orthogonalize(g.double())
    with pytest.raises(ValueError):
        sg.orthogonalize(g[0])
    with pytest.raises(ValueError):
        sg.orthogonalize(g.t()[:, :4])
    with pytest.raises(ValueError):
        sg.orthogonalize(g, coeffs=(1.0, 2.0))
    with pytest.raises(ValueError):
        sg.orthogonalize(g, out=torch.zeros(8, 8, device="cuda"))
    for kw in (dict(steps=0), dict(steps=101), dict(eps=0.0), dict(coeffs=(float("inf"), 0.0, 0.0))):
        with pytest.raises(sg.GemmError) as e:
            sg.orthogonalize(g, **kw)
        assert e.value.status == sg.GEMM_ERR_INVALID_ARG


# Both ways through the operator (a short side up to 256 stays on chip), wide and tall.
@pytest.mark.parametrize("shape", [(96, 700), (700, 96), (200, 300), (310, 420)], ids=str)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_extreme_scales_of_the_gradient(shape, dt):
    g = gradient(*shape, seed=11).to(DT[dt])
    ref = sg.orthogonalize(g.cuda())
    for k in (-105, -30, 30, 120):
        got = sg.orthogonalize((g.double() * 2.0 ** k).to(DT[dt]).cuda(), eps=1e-38)
        assert (got.double() - ref.double()).norm() <= 2.0 ** -9 * ref.double().norm(), k


@pytest.mark.parametrize("shape", [(128, 512), (129, 192), (128, 513), (193, 129), (4096, 128), (128, 4097),
                                   (256, 1536), (1537, 256), (255, 1001), (2, 4001), (4001, 100), (257, 64)], ids=str)
def test_edges_of_the_chip(shape):
    g = gradient(*shape, seed=12)
    check(sg.orthogonalize(g.cuda()), g)


@pytest.mark.parametrize("b,m,n", [(200, 20, 24), (40, 130, 200), (60, 200, 260), (30, 64, 1100), (3, 1000, 70)])
def test_many_small_matrices(b, m, n):
    gen = torch.Generator().manual_seed(b)
    g = torch.randn(b, m, n, generator=gen)
    got = sg.orthogonalize(g.cuda())
    assert torch.equal(got, sg.orthogonalize(g.cuda()))
    for i in (0, 1, b // 2, b - 1):
        check(got[i], g[i])


# The rows (or columns) of a matrix far from square have nearly equal norms,
# so that the diagonals of the products share one rounding error.  The result
# may be half as far again from the exact one as its own rounding to bf16.
@pytest.mark.parametrize("shape", [(64, 7608), (7000, 48), (40, 3000), (100, 1000), (300, 9000)], ids=str)
def test_far_from_square(shape):
    g = gradient(*shape, seed=13)
    exact = iterate(g)
    once = float((exact.bfloat16().double() - exact).norm())
    assert float((sg.orthogonalize(g.cuda()).double().cpu() - exact).norm()) <= 1.5 * once
