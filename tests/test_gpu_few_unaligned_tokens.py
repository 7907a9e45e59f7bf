"""A few tokens whose rows are not 16-byte aligned, over weights that are."""
from __future__ import annotations

import pytest
import torch

import software_pipelined_tiled_gemm_gb300 as sg
from tests.test_gpu_gated_ffn import assert_within, inputs, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    sg.check_operators()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("size", [(1, 256, 520), (8, 1024, 264), (16, 72, 1000), (27, 520, 136)], ids=str)
def test_few_unaligned_tokens_over_aligned_weights(size, dt):
    m, d, i = size
    x, w_in, w_out, _ = inputs(m, d, i, dt, seed=6)
    want = reference(x, w_in, w_out, torch.zeros_like(x), "silu", dt)["y"]
    x, w_in, w_out = x.cuda(), w_in.cuda(), w_out.cuda()
    ref = sg.gated_ffn(x, w_in, w_out)
    assert_within(ref, want, size)
    for pitch, off in ((d, 1), (d + 3, 0), (d + 8, 5), (d + 1, 7)):
        buf = torch.full((m * pitch + off,), float("nan"), dtype=x.dtype, device="cuda")
        view = buf.as_strided((m, d), (pitch, 1), off)
        view.copy_(x)
        assert torch.equal(sg.gated_ffn(view, w_in, w_out), ref), (pitch, off)


def test_unaligned_tokens_do_not_slow_the_pass_over_aligned_weights():
    # The tokens are 8 KB beside 403 MB of weights.  Reading the weights in the
    # unaligned form for their sake took 1.28 times as long.
    x, w_in, w_out, _ = (t.cuda() for t in inputs(1, 4096, 16384, "bf16", seed=7))
    odd = torch.empty(4097, dtype=x.dtype, device="cuda")[1:].view(1, 4096)
    odd.copy_(x)
    times = {}
    for _ in range(15):
        for name, tokens in (("aligned", x), ("odd", odd)):
            start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            torch.cuda.synchronize()
            start.record()
            for _ in range(10):
                sg.gated_ffn(tokens, w_in, w_out)
            end.record()
            torch.cuda.synchronize()
            times.setdefault(name, []).append(start.elapsed_time(end))
    assert min(times["odd"]) < 1.15 * min(times["aligned"]), times
