"""Calls and replayed graphs that run beside one another.

Split tiles are joined through flags and partials in a call's own workspace,
so what else runs on the device, on whatever stream, does not touch them.  The
sizes take stream-K (first products and later ones) and clusters on 152 SMs."""
from __future__ import annotations

import pytest
import torch

import software_pipelined_tiled_gemm_gb300 as sg
from tests.test_gpu_gated_ffn import inputs, run_all
from tests.test_gpu_orthogonalize import gradient

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    sg.check_operators()


def works():
    """Calls with results that a repeat gives bit for bit."""
    block = [t.cuda() for t in inputs(150, 3000, 2560, "bf16", seed=1)]     # first product stream-K
    late = [t.cuda() for t in inputs(257, 1544, 2050, "bf16", seed=2)]      # later ones, and clusters
    wide = gradient(1100, 4100, seed=3).cuda()
    return [lambda: list(run_all(*block, "silu").values()), lambda: list(run_all(*late, "gelu").values()),
            lambda: [sg.orthogonalize(wide)]]


def test_graphs_of_one_capture_stream_replayed_side_by_side():
    calls = works()
    want = [f() for f in calls]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graphs, got = [], []
    for f in calls + calls:                  # two graphs of each, all captured on one stream
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got.append(f())
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(10):
        for out in got:
            for t in out:
                t.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            for s, graph in zip(streams, graphs):
                with torch.cuda.stream(s):
                    graph.replay()
            with torch.cuda.stream(side):    # and calls on the stream that captured them
                eager = [f() for f in calls]
        torch.cuda.synchronize()
        for out, ref in list(zip(got, want + want)) + list(zip(eager, want)):
            for a, b in zip(out, ref):
                assert torch.equal(a, b)


def test_a_call_may_be_captured_on_any_stream_after_one_call_on_the_device():
    x, w_in, w_out, _ = (t.cuda() for t in inputs(70, 3000, 2560, "f16", seed=4))
    want = sg.gated_ffn(x, w_in, w_out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        got = sg.gated_ffn(x, w_in, w_out)
    got.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_flags_left_in_a_workspace_do_not_matter():
    # Workspaces come from PyTorch's allocator: one full of ones (flags that look raised).
    calls = works()
    want = [f() for f in calls]
    for _ in range(3):
        for f, ref in zip(calls, want):
            torch.cuda.synchronize()
            torch.cuda.empty_cache()
            dirty = [torch.ones(64 << 18, dtype=torch.int32, device="cuda") for _ in range(4)]
            del dirty
            for a, b in zip(f(), ref):
                assert torch.equal(a, b)
