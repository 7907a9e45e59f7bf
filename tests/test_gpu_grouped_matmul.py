"""Products grouped by expert on the GPU against their formulas in 64 bits.

Bounds.  With u half a step of the 16-bit type relative to the value (2^-8
bf16, 2^-11 fp16) and c(K) = (K + 16) 2^-23 for a K-term fp32 sum, whatever its
order, a product's error is at most c(K) times the product of the operands'
absolute values, and u times the result for its one rounding.
"""
from __future__ import annotations

import pytest
import torch

import software_pipelined_tiled_gemm_gb300 as sg

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"bf16": 1e-38, "f16": 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    sg.check_operators()


def c(k):
    return (k + 16) * 2.0 ** -23


def offsets_of(sizes, before=0):
    at = [before]
    for s in sizes:
        at.append(at[-1] + s)
    return torch.tensor(at)


def inputs(sizes, n, k, dt, seed, before=0, after=0):
    """x, w, dy and offsets; rows of no group hold NaN and infinities."""
    gen = torch.Generator().manual_seed(seed)
    off = offsets_of(sizes, before)
    rows = int(off[-1]) + after
    x = torch.randn(rows, k, generator=gen)
    dy = torch.randn(rows, n, generator=gen)
    for t in (x, dy):
        t[:before] = float("nan")
        t[int(off[-1]):] = float("inf")
    w = torch.randn(len(sizes), n, k, generator=gen) * k ** -0.5
    return x.to(DT[dt]).cuda(), w.to(DT[dt]).cuda(), dy.to(DT[dt]).cuda(), off.cuda()


def reference(x, w, dy, off, dt):
    """{name: (value, bound)}; rows of no group are 0 and exactly so."""
    u = U[dt]
    x, w, dy, ends = x.double(), w.double(), dy.double(), off.tolist()
    e, n, k = w.shape
    out = {"y": (x.new_zeros(len(x), n),) * 2, "dx": (x.new_zeros(len(x), k),) * 2, "dw": (x.new_zeros(e, n, k),) * 2}
    out = {name: tuple(t.clone() for t in pair) for name, pair in out.items()}
    for g in range(e):
        r = slice(ends[g], ends[g + 1])
        a, b, we = x[r], dy[r], w[g]
        for name, at, v, bound in (("y", r, a @ we.T, c(k) * (a.abs() @ we.abs().T)),
                                   ("dx", r, b @ we, c(n) * (b.abs() @ we.abs())),
                                   ("dw", g, b.T @ a, c(len(a)) * (b.abs().T @ a.abs()))):
            out[name][0][at] = v
            out[name][1][at] = bound + u * (v.abs() + bound) + (TINY[dt] if len(a) else 0.0)
    return out


def assert_within(got, want, what):
    value, bound = want
    assert got.shape == value.shape, what
    err = (got.double() - value).abs()
    assert bool((err <= bound).all()), (what, float((err / bound.clamp(min=1e-300)).max()))


def run_all(x, w, dy, off):
    y = sg.grouped_matmul(x, w, off)
    dx, dw = sg.grouped_matmul_backward(dy, x, w, off)
    return {"y": y, "dx": dx, "dw": dw}


SIZES = [
    ([1], 64, 64), ([1], 1, 1), ([5, 0, 3], 8, 72), ([0, 0, 1, 0], 136, 264), ([0, 0], 64, 64),
    ([17, 16, 15, 1, 33], 256, 128), ([63, 64, 65], 320, 512), ([127, 0, 129, 31], 33, 67), ([300], 1000, 257),
    ([255, 256, 257], 264, 136), ([1] * 40, 72, 200), ([513, 2, 700], 512, 640), ([64] * 8, 2048, 128),
    ([900, 0, 0, 40], 129, 1531), ([2500], 640, 96),
]


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_product_and_gradients(size, dt):
    sizes, n, k = size
    before, after = (3, 5) if n % 16 else (0, 0)
    ts = inputs(sizes, n, k, dt, sum(sizes) + n, before, after)
    want = reference(*ts, dt)
    for name, got in run_all(*ts).items():
        assert_within(got, want[name], name)
    sg.check_operators()


# Few rows a group: passes over the weights as they lie.  Shares of blocks that span several groups,
# groups without rows, more rows in a group than are held at a time, rows too long for eight tokens.
FEW = [
    ([1, 0, 1, 1], 2048, 512), ([0] * 7 + [2], 300, 1000), ([1] * 60, 16, 72), ([0, 3, 0, 0, 1], 1000, 257),
    ([9] + [0] * 7, 136, 1000), ([33] + [0] * 31 + [1], 200, 640), ([40, 1] + [0] * 20, 57, 333),
    ([2, 1], 40, 20001), ([1, 2, 0, 1], 24, 24000), ([70] + [1] * 9, 33, 129),
]


@pytest.mark.parametrize("size", FEW, ids=str)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_few_rows_a_group(size, dt):
    sizes, n, k = size
    for before, after in ((0, 0), (2, 3)):
        x, w, dy, off = inputs(sizes, n, k, dt, sum(sizes) + n, before, after)
        want = reference(x, w, dy, off, dt)["y"]
        y = sg.grouped_matmul(x, w, off)
        assert_within(y, want, before)
        assert torch.equal(y, sg.grouped_matmul(x, w, off))
        odd = torch.full((w.numel() + 8,), float("nan"), dtype=w.dtype, device="cuda")[1:1 + w.numel()].view(w.shape)
        odd.copy_(w)
        out = torch.full_like(y, 7.0)
        assert_within(sg.grouped_matmul(x, odd, off)[before:len(x) - after], tuple(t[before:len(x) - after] for t in want), "odd")
        sg.grouped_matmul(x, w, off, out=out)
        assert (out[:before] == 7).all() and (out[len(x) - after:] == 7).all()
        assert torch.equal(out[before:len(x) - after], y[before:len(x) - after])
    sg.check_operators()


def test_many_groups():
    sizes = [(i * 7) % 5 for i in range(1000)]
    ts = inputs(sizes, 40, 96, "bf16", seed=2, after=2)
    want = reference(*ts, "bf16")
    for name, got in run_all(*ts).items():
        assert_within(got, want[name], name)


def test_most_groups():
    off = torch.zeros(sg.MAX_GROUPS + 1, dtype=torch.int64, device="cuda")
    off[2000:] = 3
    x = torch.randn(4, 16, device="cuda").bfloat16()
    w = torch.randn(sg.MAX_GROUPS, 8, 16, device="cuda").bfloat16()
    dy = torch.randn(4, 8, device="cuda").bfloat16()
    want = reference(x, w, dy, off, "bf16")
    for name, got in run_all(x, w, dy, off).items():
        assert_within(got, want[name], name)
    sg.check_operators()


def test_no_rows():
    x, w, dy, off = inputs([0, 0, 0], 24, 40, "f16", seed=0)
    got = run_all(x, w, dy, off)
    assert got["y"].shape == (0, 24) and got["dx"].shape == (0, 40)
    assert got["dw"].shape == (3, 24, 40) and not got["dw"].any()


@pytest.mark.parametrize("n,k", [(64, 128), (33, 65)])
def test_pitch_and_alignment(n, k):
    """Rows with a pitch, from any 2-byte address, and outputs at odd addresses."""
    x, w, dy, off = inputs([70, 5, 200], n, k, "bf16", seed=3, before=1, after=4)
    want = reference(x, w, dy, off, "bf16")
    rows = len(x)
    for shift in (0, 1, 3):
        def wide(t):
            big = torch.full((rows, t.shape[1] + 13), float("nan"), dtype=t.dtype, device="cuda")
            big[:, shift:shift + t.shape[1]] = t
            return big[:, shift:shift + t.shape[1]]

        def odd(shape):
            size = 1
            for s in shape:
                size *= s
            return torch.full((size + 8,), float("nan"), dtype=x.dtype, device="cuda")[shift:shift + size].view(shape)
        xs, ds, ws = wide(x), wide(dy), odd(w.shape)
        ws.copy_(w)
        y, dx, dw = odd((rows, n)), odd((rows, k)), odd(w.shape)
        assert sg.grouped_matmul(xs, ws, off, out=y) is y
        got = sg.grouped_matmul_backward(ds, xs, ws, off, out=(dx, dw))
        assert got[0] is dx and got[1] is dw
        for name, t in (("y", y), ("dx", dx), ("dw", dw)):
            if name != "dw":     # given outputs keep their rows of no group
                assert t[:1].isnan().all() and t[-4:].isnan().all()
                t[:1] = 0
                t[-4:] = 0
            assert_within(t, want[name], (name, shift))


def test_each_gradient_alone():
    x, w, dy, off = inputs([40, 0, 90], 96, 72, "f16", seed=4)
    dx, dw = sg.grouped_matmul_backward(dy, x, w, off)
    a, none = sg.grouped_matmul_backward(dy, x, w, off, need=(True, False))
    assert none is None and torch.equal(a, dx)
    none, b = sg.grouped_matmul_backward(dy, x, w, off, need=(False, True))
    assert none is None and torch.equal(b, dw)
    assert sg.grouped_matmul_backward(dy, x, w, off, need=(False, False)) == (None, None)


@pytest.mark.parametrize("groups", [2, 5])      # tiles, and passes over the weights
@pytest.mark.parametrize("off", [[0, 4, 3], [-1, 4, 8], [0, 4, 9], [2, 1, 8], [0, 1 << 40, 8]])
def test_wrong_offsets_are_reported_and_write_nothing(off, groups):
    off = off + off[-1:] * (groups - 2)
    x = torch.randn(8, 64, device="cuda").bfloat16()
    w = torch.randn(groups, 32, 64, device="cuda").bfloat16()
    dy = torch.randn(8, 32, device="cuda").bfloat16()
    off = torch.tensor(off, device="cuda")
    y, dx, dw = (torch.full_like(t, 7.0) for t in (dy, x, w))
    for call in (lambda: sg.grouped_matmul(x, w, off, out=y),
                 lambda: sg.grouped_matmul_backward(dy, x, w, off, out=(dx, dw))):
        call()
        with pytest.raises(sg.GemmError, match="offsets"):
            sg.check_operators()
    assert (y == 7).all() and (dx == 7).all() and (dw == 7).all()
    sg.check_operators()


def test_repeats_bit_for_bit_and_against_differences():
    x, w, dy, off = inputs([100, 33, 280], 256, 192, "bf16", seed=5)
    first, again = run_all(x, w, dy, off), run_all(x, w, dy, off)
    for name in first:
        assert torch.equal(first[name], again[name]), name
    # <dy, y(x + h d)> - <dy, y(x)> = h <dx, d> for the linear product: differences of the operator itself.
    d = torch.randn(x.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).bfloat16()
    y1 = sg.grouped_matmul(d, w, off)
    left, right = (dy.double() * y1.double()).sum(), (first["dx"].double() * d.double()).sum()
    scale = (dy.double().abs() * y1.double().abs()).sum() + (first["dx"].double().abs() * d.double().abs()).sum()
    assert abs(left - right) <= (2.0 ** -8 + c(256)) * scale


def test_streams_and_graph():
    x, w, dy, off = inputs([100, 0, 333], 264, 320, "bf16", seed=6, after=3)
    want = run_all(x, w, dy, off)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run_all(x, w, dy, off)
    side.synchronize()
    for name in want:
        assert torch.equal(got[name], want[name]), name
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run_all(x, w, dy, off)
    # The groups' sizes may change from replay to replay.
    new_off = torch.tensor([0, 0, 250, 400], device="cuda")
    new = inputs([0, 250, 150], 264, 320, "bf16", seed=7, after=36)
    expect = run_all(new[0], new[1], new[2], new_off)
    x.copy_(new[0]), w.copy_(new[1]), dy.copy_(new[2]), off.copy_(new_off)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for name in expect:
        assert torch.equal(held[name], expect[name]), name
    sg.check_operators()
