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
