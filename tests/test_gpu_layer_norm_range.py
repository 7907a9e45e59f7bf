"""Layer norm of rows at the ends of fp32's range, against the formulas in 64 bits.

The bounds are those of test_gpu_layer_norm.py: they are relative to a row's own
sizes, so they hold at any of them.
"""
from __future__ import annotations

import pytest
import torch

import software_pipelined_tiled_gemm_gb300 as sg
from tests.test_gpu_layer_norm import DT, assert_within, reference

pytestmark = pytest.mark.gpu

COLS = [40, 1000, 1531, 4096, 4099, 9000, 30000, 33000]
MOST = 3.3e38   # below the largest bf16 and the largest fp32


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    sg.check_operators()


def odd(t):
    """The same values where no row allows 16-byte vectors."""
    flat = torch.full((t.numel() + 16,), float("nan"), dtype=t.dtype, device="cuda")
    flat[1:1 + t.numel()] = t.reshape(-1)
    return flat[1:1 + t.numel()].view(t.shape)


def normal(*shape, seed=1):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("size", [3e36, 1e37, 3e37])
def test_sums_beyond_the_range(cols, dt, size):
    """The differences are finite, their sum is not."""
    x = (normal(6, cols) * size).to(DT[dt])
    want = reference(x, None, None, x)["y"]
    for t in (x, odd(x)):
        assert_within(sg.layer_norm(t), want, size)


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_differences_beyond_the_range(cols, dt):
    """Rows at both ends of the range: a mean near one of them and an element at the other."""
    x = torch.full((4, cols), -MOST, device="cuda")
    x[0, 0] = x[1, -1] = x[2, cols // 2] = MOST
    x[3, :cols // 3] = MOST
    x = x.to(DT[dt])
    want = reference(x, None, None, x)["y"]
    for t in (x, odd(x)):
        assert_within(sg.layer_norm(t), want, "y")


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_gradients_of_rows_beyond_the_range(cols, dt):
    x = torch.cat([normal(4, cols) * 3e37, torch.full((3, cols), -MOST, device="cuda")])
    x[4, 0] = x[5, -1] = x[6, cols // 2] = MOST
    x, dy = x.to(DT[dt]), (normal(7, cols, seed=2) * 1e33).to(DT[dt])
    want = reference(x, None, None, dy)
    for place in (lambda t: t, odd):
        y, kept = sg.layer_norm(place(x), save=True)
        got = sg.layer_norm_backward(place(dy), place(x), None, kept)
        for name, t in zip(("dx", "dweight", "dbias"), got):
            assert_within(t, want[name], name)


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_constant_rows(cols, dt):
    """x - mean is 0 and the variance is 0, however large x is and whatever n x rounds to:
    y is the bias, rstd 1 / sqrt(eps), and dx rstd (dy - <dy>).

    h is 0 to the bit where the mean's rounding, d = x - mean, is the larger part of
    var + eps.  Elsewhere |d| is at most sqrt(eps), in all columns the same, so low is d
    but for its sum's error, c(n) |d|, and |h| = |d - low| rstd at most c(n)."""
    top = 65000.0 if dt == "f16" else MOST
    sizes = [1.5, -777.0, 64996.0] + [-10.0 ** e for e in range(6, 39, 4)] + [1e27, 3.3e28, 1e30, 1e37, MOST, -MOST]
    x = torch.tensor(sizes, device="cuda").clamp(-top, top).to(DT[dt])[:, None].expand(-1, cols).contiguous()
    b, dy = normal(cols).to(DT[dt]), (normal(len(sizes), cols, seed=2) + 0.5).to(DT[dt])
    g = dy.double()
    mean, size = g.mean(1, keepdim=True), g.abs().mean(1, keepdim=True)
    rstd = 1e-5 ** -0.5
    # The mean's sum, the difference, the products with rstd, and rstd itself (2^-21).
    c = (max(32, cols / 1024) + 48) * 2.0 ** -23
    bound = rstd * ((c + 2.0 ** -22) * size + 2.0 ** -20 * (g.abs() + mean.abs()) + c * c * size)
    value = rstd * (g - mean)
    u = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dt]
    bound = bound + u * (value.abs() + bound)
    for place in (lambda t: t, odd):
        y, kept = sg.layer_norm(place(x), None, b, save=True)
        near = c + 2.0 ** -23 * b.double().abs()
        assert bool(((y.double() - b.double()).abs() <= near + u * (b.double().abs() + near)).all())
        far = x[:, 0].abs() > 1e9   # d is 0 or at least 2^-24 x
        assert torch.equal(y[far], b.expand_as(y)[far])
        assert bool((kept.stats[2].double() / rstd - 1).abs().max() <= 2.0 ** -21)
        dx = sg.layer_norm_backward(place(dy), place(x), None, kept, need=(True, False, False))[0]
        assert_within(dx, (value, bound), "dx")


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_without_eps(cols, dt):
    """Squares below fp32's range, which eps does not hide."""
    x = (normal(4, cols) * torch.tensor([[1e-18], [1e-21], [1e-30], [1e-37]], device="cuda")).to(DT[dt])
    dy = (normal(4, cols, seed=2) * 1e-10).to(DT[dt])
    want = reference(x, None, None, dy, eps=0.0)
    for place in (lambda t: t, odd):
        y, kept = sg.layer_norm(place(x), eps=0.0, save=True)
        assert_within(y, want["y"], "y")
        got = sg.layer_norm_backward(place(dy), place(x), None, kept)
        for name, t in zip(("dx", "dweight", "dbias"), got):
            assert_within(t, want[name], name)


@pytest.mark.parametrize("cols", [64, 1024, 8192])   # (sums of equal numbers are exact)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_gradient_of_unaligned_rows_whose_mean_is_large(cols, dt):
    """What a row's first and last vector hold beside the row is no part of it, nor is its distance from the mean."""
    x = torch.full((9, cols), 2.0 ** 121, device="cuda").to(DT[dt])
    dy = (normal(9, cols, seed=2) + 0.5).to(DT[dt])
    y, kept = sg.layer_norm(x, save=True)
    want = sg.layer_norm_backward(dy, x, None, kept, need=(True, False, False))[0]
    assert bool(torch.isfinite(want).all())
    y, kept = sg.layer_norm(odd(x), save=True)
    dx = sg.layer_norm_backward(odd(dy), odd(x), None, kept, need=(True, False, False))[0]
    # Sums in another order: c(n) of |dy|, and a rounding of the output.
    bound = 317.0 * (max(32, cols / 1024) + 48) * 2.0 ** -22 * dy.double().abs().mean(1, keepdim=True)
    u = {"f32": 2.0 ** -23, "bf16": 2.0 ** -7}[dt]
    assert_within(dx, (want.double(), bound + u * (want.double().abs() + bound)), "dx")


@pytest.mark.parametrize("cols", [13, 61, 1019, 1531, 4099, 33000])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_such_rows_between_others(cols, dt):
    """Each row by itself: rows of every kind in one matrix, out of place and in place."""
    x = normal(64, cols) * 2 + 1
    x[1::8] *= 3e37
    x[2::8] = 1e30
    x[3::8, cols // 2] = float("nan")
    x[4::8, 0] = float("inf")
    x[5::8] = x[5::8] * 1e-3 + 1e4
    x[6::8] = 0.0
    x = x.to(DT[dt])
    # (One of the random rows of 33000 columns reaches beyond 3.4e38 and holds an infinity.)
    whole = torch.isfinite(x).all(1)
    assert not whole[3::8].any() and not whole[4::8].any() and int(whole.sum()) >= 47
    # (A row of 1e30 or of zeros: its h is 0 to the bit, which the general bound does not ask for.)
    value, bound = reference(x[whole], None, None, x[whole])["y"]
    for t in (x, odd(x)):
        y = sg.layer_norm(t)
        assert_within(y[whole], (value, bound), "y")
        assert y[~whole].isnan().all() and not y[2::8].any() and not y[6::8].any()
        assert torch.equal(sg.layer_norm(t, out=t)[whole], y[whole])


@pytest.mark.parametrize("cols", [5, 40, 1000, 4099, 9000, 33000])
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("eps", [1e-5, 0.0, 1e-30])
def test_nan_and_infinities_beside_anything(cols, dt, eps):
    """One of them makes its whole row NaN, whatever the others are: zeros, subnormal or large numbers."""
    top = 6e4 if dt == "f16" else MOST
    rows = [0.0, 1e-38, 1e-40, -1e-30, 1e-7, 1.0, top]
    marks = [float("nan"), float("inf"), float("-inf")]
    x = torch.tensor(rows, device="cuda").repeat(len(marks))[:, None].expand(-1, cols).to(DT[dt]).contiguous()
    for i in range(len(x)):
        x[i, (i * 7) % cols] = marks[i // len(rows)]
    both = torch.zeros(1, cols, device="cuda", dtype=DT[dt])
    both[0, 0], both[0, -1] = float("inf"), float("-inf")
    x = torch.cat([x, both, torch.full_like(both, float("nan")), torch.full_like(both, float("inf"))])
    dy = normal(len(x), cols, seed=2).to(DT[dt])
    for place in (lambda t: t, odd):
        y, kept = sg.layer_norm(place(x), eps=eps, save=True)
        assert y.isnan().all()
        assert sg.layer_norm_backward(place(dy), place(x), None, kept, need=(True, False, False))[0].isnan().all()
