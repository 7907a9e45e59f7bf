"""The first call of an operator in a process: what it sets up is set up on any
stream, in a capture, and for several threads at once."""
from __future__ import annotations

import os
import subprocess
import sys
import textwrap

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def child(code):
    out = subprocess.run([sys.executable, "-c", textwrap.dedent(code)], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert out.returncode == 0, out.stderr[-4000:]
    return out.stdout


@pytest.mark.gpu
def test_first_layer_norm_in_a_capture():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    assert "same" in child("""
        import torch
        import software_pipelined_tiled_gemm_gb300 as sg
        x = torch.randn(300, 4096, device="cuda").bfloat16()
        sg.token_logprobs(x)              # the handle
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y, kept = sg.layer_norm(x, save=True)
            dx = sg.layer_norm_backward(y, x, None, kept, need=(True, False, False))[0]
        graph.replay()
        torch.cuda.synchronize()
        want, kept = sg.layer_norm(x, save=True)
        assert torch.equal(y, want) and float(want.float().abs().max()) > 1
        assert torch.equal(dx, sg.layer_norm_backward(want, x, None, kept, need=(True, False, False))[0])
        sg.check_operators()
        print("same")
    """)


@pytest.mark.gpu
def test_first_layer_norms_of_threads():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    assert "same" in child("""
        import threading
        import torch
        import software_pipelined_tiled_gemm_gb300 as sg
        xs = [torch.randn(64, 16384, device="cuda").to(t) for t in (torch.bfloat16, torch.float32, torch.float16)]
        torch.cuda.synchronize()
        got, go = [None] * 3, threading.Barrier(3)
        def run(i):
            with torch.cuda.stream(torch.cuda.Stream()):
                go.wait()
                got[i] = sg.layer_norm(xs[i])
                torch.cuda.current_stream().synchronize()
        threads = [threading.Thread(target=run, args=(i,)) for i in range(3)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert all(torch.equal(g, sg.layer_norm(x)) for g, x in zip(got, xs))
        sg.check_operators()
        print("same")
    """)
