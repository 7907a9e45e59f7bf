"""Refusals and device-side errors of the grouped products, layer norm and AdamW, and
calls of them that run beside one another."""
from __future__ import annotations

import time

import pytest
import torch

import software_pipelined_tiled_gemm_gb300 as sg
from software_pipelined_tiled_gemm_gb300 import operators
from tests import test_gpu_adamw, test_gpu_grouped_matmul, test_gpu_layer_norm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    sg.check_operators()


@pytest.mark.parametrize("which", range(3))
def test_timeout_is_reported_and_the_next_call_is_right(which):
    """The hook leaves one copy out; the waits run out after their limit and nothing faults or hangs."""
    dev = torch.device("cuda", 0)
    x, w, dy, off = test_gpu_grouped_matmul.inputs([300, 0, 700], 520, 264, "bf16", seed=1)
    call = (lambda: sg.grouped_matmul(x, w, off),
            lambda: sg.grouped_matmul_backward(dy, x, w, off, need=(True, False))[0],
            lambda: sg.grouped_matmul_backward(dy, x, w, off, need=(False, True))[1])[which]
    want = call()
    sg.check_operators()
    try:
        operators._configure(dev, timeout_ns=20_000_000, debug_fault=1)
        t0 = time.perf_counter()
        call()
        with pytest.raises(sg.GemmError) as e:
            sg.check_operators()
        assert e.value.status == sg.GEMM_ERR_TIMEOUT
        assert time.perf_counter() - t0 < 20.0
    finally:
        operators._configure(dev)
    got = call()
    sg.check_operators()
    assert torch.equal(got, want)


def test_graphs_and_calls_side_by_side():
    """Replays of graphs captured on one stream, on streams of their own, beside eager calls."""
    mul = test_gpu_grouped_matmul.inputs([300, 5, 700, 64], 520, 264, "bf16", seed=2)
    few = test_gpu_grouped_matmul.inputs([1, 0, 2, 1], 520, 264, "bf16", seed=3)
    ragged = test_gpu_grouped_matmul.inputs([30, 5], 33, 65, "f16", seed=4)
    norm = test_gpu_layer_norm.inputs(500, 1544, "bf16", "f32", seed=5)
    calls = [lambda: list(test_gpu_grouped_matmul.run_all(*mul).values()),
             lambda: list(test_gpu_grouped_matmul.run_all(*few).values()),
             lambda: list(test_gpu_grouped_matmul.run_all(*ragged).values()),
             lambda: list(test_gpu_layer_norm.run_all(*norm).values())]
    want = [f() for f in calls]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graphs, got = [], []
    for f in calls + calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            # (torch.equal inside run_all would wait for the device)
            got.append(capture(f, mul, few, ragged, norm, calls))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for out in got:
            for t in out:
                t.zero_()
        torch.cuda.synchronize()
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        with torch.cuda.stream(side):
            eager = [capture(f, mul, few, ragged, norm, calls) for f in calls]
        torch.cuda.synchronize()
        for out, ref in list(zip(got, want + want)) + list(zip(eager, want)):
            for a, b in zip(out, ref):
                assert torch.equal(a, b)


def capture(f, mul, few, ragged, norm, calls):
    i = calls.index(f)
    if i < 3:
        return list(test_gpu_grouped_matmul.run_all(*(mul, few, ragged)[i]).values())
    x, w, b, dy = norm
    y, kept = sg.layer_norm(x, w, b, eps=test_gpu_layer_norm.EPS, save=True)
    return [y] + list(sg.layer_norm_backward(dy, x, w, kept))


def test_two_adamw_steps_on_two_streams():
    """Different tensors and states; each as if it ran alone."""
    a = [test_gpu_adamw.Case(test_gpu_adamw.SHAPES, grad="bf16", copy="bf16", bits=b, seed=20) for b in (8, 32)]
    b = [test_gpu_adamw.Case(test_gpu_adamw.SHAPES, grad="bf16", copy="bf16", bits=b, seed=20) for b in (8, 32)]
    for c in a:
        for _ in range(4):
            sg.adamw(c.params, c.grads, c.state, 1e-2, copies=c.copies)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in b]
    for _ in range(4):
        for c, s in zip(b, streams):
            with torch.cuda.stream(s):
                sg.adamw(c.params, c.grads, c.state, 1e-2, copies=c.copies)
    torch.cuda.synchronize()
    for x, y in zip(a, b):
        for p, q in zip(x.params + x.copies + list(x.state[1:3]), y.params + y.copies + list(y.state[1:3])):
            assert torch.equal(p.float(), q.float())


def test_refusals_of_grouped_products():
    x, w, dy, off = test_gpu_grouped_matmul.inputs([3, 5], 24, 40, "bf16", seed=6)
    y = sg.grouped_matmul(x, w, off)

    def refuse(error, match, f, *args, **kw):
        with pytest.raises(error, match=match):
            f(*args, **kw)
    mul, back = sg.grouped_matmul, sg.grouped_matmul_backward
    refuse(TypeError, "x must", mul, x.float(), w, off)
    refuse(TypeError, "same dtype", mul, x, w.half(), off)
    refuse(ValueError, "columns", mul, x[:, :8], w, off)
    refuse(ValueError, "w must", mul, x, w[0], off)
    refuse(ValueError, "w must", mul, x, w.mT, off)
    refuse(ValueError, "w must", mul, x, w[:0], off[:1])
    refuse(ValueError, "matrix", mul, x[None], w, off)
    refuse(ValueError, "x must be contiguous", mul, x.t().contiguous().t(), w, off)
    refuse(TypeError, "int64", mul, x, w, off.int())
    refuse(ValueError, "offsets", mul, x, w, off[:2])
    refuse(ValueError, "CUDA", mul, x, w, off.cpu())
    refuse(ValueError, "out", mul, x, w, off, out=y.float())
    refuse(ValueError, "out", mul, x, w, off, out=y[:4])
    refuse(sg.GemmError, "overlaps", mul, x, w, off, out=w.view(-1)[:y.numel()].view(y.shape))
    refuse(ValueError, "dy", back, dy[:4], x, w, off)
    refuse(sg.GemmError, "overlaps", back, dy, x, w, off, out=(x, None))
    buf = torch.empty(w.numel(), dtype=x.dtype, device="cuda")
    refuse(sg.GemmError, "overlaps", back, dy, x, w, off, out=(buf[:x.numel()].view(x.shape), buf.view(w.shape)))


def test_refusals_of_layer_norm():
    x, w, b, dy = test_gpu_layer_norm.inputs(6, 40, "bf16", "bf16", seed=7)
    y, kept = sg.layer_norm(x, w, b, save=True)

    def refuse(error, match, f, *args, **kw):
        with pytest.raises(error, match=match):
            f(*args, **kw)
    norm, back = sg.layer_norm, sg.layer_norm_backward
    refuse(TypeError, "x must", norm, x.double())
    refuse(ValueError, "weight", norm, x, w[:8])
    refuse(TypeError, "weight", norm, x, w.half())
    refuse(TypeError, "same dtype", norm, x, w, b.float())
    refuse(ValueError, "eps", norm, x, w, b, eps=-1.0)
    refuse(ValueError, "eps", norm, x, w, b, eps=float("nan"))
    refuse(ValueError, "column", norm, x[:, :0])
    refuse(ValueError, "CUDA", norm, x, w.cpu())
    refuse(ValueError, "out", norm, x, w, b, out=y.half())
    refuse(sg.GemmError, "overlaps", norm, x[1:], w, b, out=x[:-1])
    refuse(TypeError, "kept", back, dy, x, w, None)
    refuse(ValueError, "kept", back, dy[:4], x[:4], w, kept)
    refuse(ValueError, "dy", back, dy[:4], x, w, kept)
    refuse(sg.GemmError, "overlaps", back, dy, x, w, kept, out=(x, None, None))
    refuse(sg.GemmError, "overlaps", back, dy, x, w, kept, out=(None, w, None))


def test_large_offsets_into_memory():
    """Rows whose elements lie beyond 2^31 from the first, in each operator."""
    cols = 1 << 21
    rows = (1 << 31) // cols + 3
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_()
    y, kept = sg.layer_norm(x, save=True)
    back = sg.layer_norm_backward(y, x, None, kept, need=(True, False, False))[0]
    for r in (0, rows - 1):
        want = test_gpu_layer_norm.reference(x[r:r + 1], None, None, y[r:r + 1])
        test_gpu_layer_norm.assert_within(y[r:r + 1], want["y"], r)
        test_gpu_layer_norm.assert_within(back[r:r + 1], want["dx"], r)
    del y, back, kept
    # A weight of more than 2^31 elements in all; rows of its last groups.
    e, n, k = 260, 2056, 4096
    w = x.view(-1)[:e * n * k].view(e, n, k) if e * n * k <= x.numel() else torch.empty(e, n, k, dtype=x.dtype, device="cuda").normal_()
    t = 300
    off = torch.zeros(e + 1, dtype=torch.int64, device="cuda")
    off[e - 1:] = 20
    off[e] = t
    rows_x = torch.randn(t, k, device="cuda").bfloat16()
    got = sg.grouped_matmul(rows_x, w, off)
    bound = test_gpu_grouped_matmul.c(k)
    for g, s in ((e - 2, slice(0, 20)), (e - 1, slice(20, t))):
        a, b = rows_x[s].double(), w[g].double()
        value, err = a @ b.T, bound * (a.abs() @ b.abs().T)
        test_gpu_grouped_matmul.assert_within(got[s], (value, err + 2.0 ** -8 * (value.abs() + err) + 1e-38), g)
    sg.check_operators()
