"""Grouped products, layer norm and AdamW where an element's offset passes 32 bits:
the last rows of matrices of more than 2^32 elements.

Bounds.  A sum of n products in fp32 is off by at most n 2^-23 times the sum of
their absolute values, and its one rounding to bf16 by 2^-8 of the value.
"""
from __future__ import annotations

import pytest
import torch

import software_pipelined_tiled_gemm_gb300 as sg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.get_device_properties(0).total_memory < 120 << 30:
        pytest.skip("needs 120 GB")
    yield
    sg.check_operators()
    torch.cuda.empty_cache()


def assert_product(got, a, b):
    """got = a b^T, bf16."""
    a, b = a.double(), b.double()
    value, size = a @ b.T, a.abs() @ b.abs().T
    err = (got.double() - value).abs()
    bound = a.shape[1] * 2.0 ** -23 * size
    assert bool((err <= bound + 2.0 ** -8 * (value.abs() + bound)).all())


@pytest.mark.parametrize("each", [1, 10])   # passes over the weights, tiles
def test_grouped_products(each):
    groups, n, k = 68, 8192, 8192
    assert groups * n * k > 1 << 32
    gen = torch.Generator(device="cuda").manual_seed(1)
    w = torch.empty(groups, n, k, dtype=torch.bfloat16, device="cuda")
    w[:-1] = float("nan")   # (of the groups before, whose rows are not looked at)
    w[-1].copy_(torch.randn(n, k, generator=gen, device="cuda"))
    x = torch.randn(groups * each, k, generator=gen, device="cuda").bfloat16()
    dy = torch.randn(groups * each, n, generator=gen, device="cuda").bfloat16()
    offsets = torch.arange(groups + 1, device="cuda") * each
    last = slice((groups - 1) * each, None)
    assert_product(sg.grouped_matmul(x, w, offsets)[last], x[last], w[-1])
    dx, dw = sg.grouped_matmul_backward(dy, x, w, offsets)
    assert_product(dx[last], dy[last], w[-1].T)
    assert_product(dw[-1], dy[last].T, x[last].T)


def test_grouped_rows():
    rows, n, k = (1 << 20) + 5, 4104, 64
    assert rows * n > 1 << 32
    gen = torch.Generator(device="cuda").manual_seed(2)
    w = torch.randn(2, n, k, generator=gen, device="cuda").bfloat16()
    x = torch.randn(rows, k, generator=gen, device="cuda").bfloat16()
    offsets = torch.tensor([0, rows - 300, rows - 3], device="cuda")
    y = sg.grouped_matmul(x, w, offsets)
    last = slice(rows - 300, rows - 3)
    assert_product(y[last], x[last], w[1])
    assert not y[-3:].any()
    dx = sg.grouped_matmul_backward(y, x, w, offsets, need=(True, False))[0]
    assert_product(dx[last], y[last], w[1].T)


@pytest.mark.parametrize("cols", [4096, 4099])
def test_layer_norm(cols):
    rows = (1 << 20) + 4096
    assert rows * cols > 1 << 32
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-64:] = torch.randn(64, cols, generator=gen, device="cuda").bfloat16()
    w = torch.randn(cols, generator=gen, device="cuda")
    y, kept = sg.layer_norm(x, w, save=True)
    dx = sg.layer_norm_backward(x, x, w, kept, need=(True, False, False))[0]
    small = x[-64:].clone()   # 64 rows: they begin in the same places of 16 bytes
    y_small, kept_small = sg.layer_norm(small, w, save=True)
    assert torch.equal(y[-64:], y_small)
    assert torch.equal(kept.stats[:, -64:], kept_small.stats)
    assert torch.equal(dx[-64:], sg.layer_norm_backward(small, small, w, kept_small, need=(True, False, False))[0])


def test_adamw():
    n, tail = (1 << 32) + 1001, 1001
    gen = torch.Generator(device="cuda").manual_seed(4)
    p = torch.zeros(n, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    p[-tail:] = torch.randn(tail, generator=gen, device="cuda")
    g[-tail:] = torch.randn(tail, generator=gen, device="cuda").bfloat16()
    p_small, g_small = p[-tail:].clone(), g[-tail:].clone()
    state, state_small = sg.adamw_state([p]), sg.adamw_state([p_small])
    for _ in range(2):
        sg.adamw([p], [g], state, 1e-3)
        sg.adamw([p_small], [g_small], state_small, 1e-3)
    assert torch.equal(p[-tail:], p_small)
    assert not p[:256].any() and int(state.step) == 2
    assert torch.equal(state.exp_avg[-1024:], state_small.exp_avg)
    assert torch.equal(state.exp_avg_sq[-1024:], state_small.exp_avg_sq)
