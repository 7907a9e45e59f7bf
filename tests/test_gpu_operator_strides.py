"""Tensors with a single row or column, whose stride along it means nothing."""
from __future__ import annotations

import pytest
import torch

import software_pipelined_tiled_gemm_gb300 as sg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    sg.check_operators()


def test_one_column():
    base = torch.randn(3, 40, generator=torch.Generator().manual_seed(1)).cuda()
    column = base.t()[::2, :1]                      # 20 x 1, strides (2, 40)
    assert not column.is_contiguous() and column.stride() == (2, 40)
    assert torch.equal(sg.orthogonalize(column), sg.orthogonalize(column.contiguous()))
    assert torch.equal(sg.token_logprobs(column).lse, column[:, 0])
    x = base.bfloat16().t()[::2, :1]
    w_in, w_out = torch.ones(48, 1).bfloat16().cuda(), torch.ones(1, 24).bfloat16().cuda()
    assert torch.equal(sg.gated_ffn(x, w_in, w_out), sg.gated_ffn(x.contiguous(), w_in, w_out))


def test_one_row_of_each_matrix():
    base = torch.randn(5, 64, generator=torch.Generator().manual_seed(2)).cuda()
    rows = base.as_strided((5, 1, 60), (64, 3, 1))  # the stride between rows of one row
    assert torch.equal(sg.orthogonalize(rows), sg.orthogonalize(rows.contiguous()))


def test_rows_that_are_not_contiguous_are_still_refused():
    base = torch.randn(8, 8, device="cuda")
    for t in (base[:, ::2], base.t()[:, :2]):
        with pytest.raises(ValueError):
            sg.orthogonalize(t)
        with pytest.raises(ValueError):
            sg.token_logprobs(t)
    with pytest.raises(ValueError):
        sg.orthogonalize(base.as_strided((8, 4), (2, 1)))     # rows that overlap
