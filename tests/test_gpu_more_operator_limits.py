"""What the grouped products and layer norm refuse before they launch anything: sizes that
their index arithmetic does not hold, and kept statistics of another layout."""
from __future__ import annotations

import ctypes

import pytest
import torch

import software_pipelined_tiled_gemm_gb300 as sg
from software_pipelined_tiled_gemm_gb300 import operators

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    sg.check_operators()


@pytest.mark.parametrize("backward", [0, 1])
def test_rows_that_32_bits_do_not_count(backward):
    """Rows up to the next tile, and up to the next of a launch's warps, stay below 2^31."""
    handle = operators._handle(torch.device("cuda", 0))
    where = torch.zeros(64, dtype=torch.int64, device="cuda")
    need = ctypes.c_size_t()

    def status(rows):
        p = where.data_ptr()
        a = sg.GroupedArgs(rows, 3, 64, 64, 1, p, p, 64, p, p, 0, p, 64, p, p)
        return operators._lib().gemm_grouped_workspace(handle, ctypes.byref(a), backward, ctypes.byref(need))
    assert status((1 << 31) - 65536) == 0
    for rows in ((1 << 31) - 65535, (1 << 31) - 256, (1 << 31) - 1, 1 << 31, 1 << 40):
        assert status(rows) == sg.GEMM_ERR_INVALID_ARG
        assert "rows" in sg.gemm_last_error()


@pytest.mark.parametrize("rows,cols", [(6, 40), (200, 1531)])
def test_kept_statistics_of_another_layout(rows, cols):
    """The kernels read three rows of fp32; a slice of them for a part of the rows is another layout."""
    x = torch.randn(rows, cols, device="cuda")
    y, kept = sg.layer_norm(x, save=True)
    half = rows // 2
    for stats in (kept.stats[:, :half], kept.stats[:2], kept.stats.half(), kept.stats.t().contiguous(), kept.stats.view(-1),
                  kept.stats.cpu(), None, torch.empty(3, 2 * rows, device="cuda")[:, ::2]):
        with pytest.raises(ValueError, match="kept"):
            sg.layer_norm_backward(y, x, None, kept._replace(stats=stats))
    with pytest.raises(ValueError, match="kept"):
        sg.layer_norm_backward(y[:half], x[:half], None, kept._replace(stats=kept.stats[:, :half], rows=half))
    # A copy of the slice has the layout.
    part = sg.LayerNormKept(kept.stats[:, :half].contiguous(), half, cols, x.dtype)
    dx = sg.layer_norm_backward(y[:half], x[:half], None, part, need=(True, False, False))[0]
    assert torch.equal(dx, sg.layer_norm_backward(y, x, None, kept, need=(True, False, False))[0][:half])
