"""What the operators ask of the allocator besides their outputs."""
from __future__ import annotations

import ctypes

import pytest
import torch

import software_pipelined_tiled_gemm_gb300 as sg
from software_pipelined_tiled_gemm_gb300 import operators
from tests.test_gpu_gated_ffn import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    sg.check_operators()


def ffn_workspace(m, d, i, backward=0):
    x, w_in, w_out, _ = (t.cuda() for t in inputs(m, d, i, "bf16", seed=1))
    lib = operators._lib()
    a = operators._ffn_args(x, w_in, w_out, "silu")
    y = torch.empty_like(x)
    a.y = a.dy = y.data_ptr()
    if backward:
        kept = torch.empty(lib.gemm_ffn_kept_bytes(m, i), dtype=torch.uint8, device="cuda")
        a.kept = kept.data_ptr()
    n = ctypes.c_size_t()
    assert lib.gemm_ffn_workspace(operators._handle(x.device), ctypes.byref(a), backward, ctypes.byref(n)) == 0
    return n.value


def test_passes_over_the_weights_take_no_room_for_partials():
    # H alone: m rows of d_inner 16-bit elements, to the next 256 bytes.
    assert ffn_workspace(1, 256, 1000) == 2048
    assert ffn_workspace(7, 264, 520) == -(-7 * 520 * 2 // 256) * 256


def test_products_on_tiles_do():
    partials = 152 * 128 * 256 * 4
    assert ffn_workspace(200, 256, 320) >= partials and ffn_workspace(1, 256, 320, backward=1) >= partials
