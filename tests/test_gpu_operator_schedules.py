"""The block products' schedules on the GPU against 64 bits.

Which schedule a product takes follows from its extents (run_block in
ops_api.cu).  The sizes here are chosen so that, on 152 SMs and 76 pairs, every
schedule runs in every kind of product that can take it; the comments name
them by kind: gated and gated backward, NT, NN and TN (plain; symmetric in an
update), and the updates' products with a diagonal.  Bounds are those of
test_gpu_gated_ffn.py and test_gpu_orthogonalize.py; the 64-bit results are
computed on the GPU, where products of these sizes take well under a second.
"""
from __future__ import annotations

import pytest
import torch

import software_pipelined_tiled_gemm_gb300 as sg
from tests.test_gpu_gated_ffn import inputs, reference, run_all
from tests.test_gpu_orthogonalize import gradient, iterate

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    sg.check_operators()


def check_block(size, act, dt, repeats):
    ts = [t.cuda() for t in inputs(*size, dt, seed=sum(size))]
    got = run_all(*ts, act)
    for name, (value, bound) in reference(*ts, act, dt).items():
        worst = float(((got[name].double() - value).abs() / bound).max())
        assert worst <= 1.0, (size, name, worst)
    for _ in range(repeats):
        again = run_all(*ts, act)
        for name in got:
            assert torch.equal(again[name], got[name]), (size, name)


def check_update(m, n, repeats):
    g = gradient(m, n, seed=m + n).cuda()
    got = sg.orthogonalize(g)
    exact, model = iterate(g), iterate(g, rounded=True)
    off = float((got.double() - exact).norm() / exact.norm())
    tol = 1.5 * float((model - exact).norm() / exact.norm()) + 2.0 ** -9
    assert off <= tol, (m, n, off, tol)
    for _ in range(repeats):
        assert torch.equal(sg.orthogonalize(g), got), (m, n)


# K shared by a cluster: the CTAs' partials meet in shared memory, and every
# warp stores rows that others staged.
CLUSTER = [
    (40, 1544, 72),       # gated and gated backward over 4 CTAs
    (40, 264, 1408),      # NT and NN over 4
    (40, 2056, 2560),     # gated over 2
    (150, 2056, 2560),    # gated backward over 2
    (257, 1544, 1000),    # NN over 2
    (257, 1544, 2050),    # NT over 2
    (1537, 264, 72),      # TN over 4
    (2050, 3000, 72),     # TN over 2
]


@pytest.mark.parametrize("size", CLUSTER, ids=str)
@pytest.mark.parametrize("act,dt", [("silu", "bf16"), ("gelu", "f16")])
def test_blocks_whose_k_is_shared_by_a_cluster(size, act, dt):
    check_block(size, act, dt, repeats=20)


@pytest.mark.parametrize("shape", [(260, 1200), (1200, 260), (1100, 1800), (1800, 1100)], ids=str)
def test_updates_whose_k_is_shared_by_a_cluster(shape):
    check_update(*shape, repeats=20)     # X X^T (NT) and X^T X (TN), over 4 and over 2


# Stream-K (a tile's K shared out through the workspace), more tiles than
# walkers, CTA pairs, and one or two epilogue warps a lane quarter.
LARGE = [
    (150, 3000, 2560),    # gated: stream-K on single CTAs, fewer tiles than walkers
    (900, 2056, 2560),    # gated: pairs, waves of tiles, one epilogue warp a quarter
    (900, 2304, 2560),    # gated: pairs, the last waves stream-K
    (2600, 264, 1408),    # gated: pairs, two warps over waves of tiles
    (2050, 3000, 520),    # gated backward: stream-K on single CTAs
    (2600, 264, 3200),    # gated backward: pairs, waves of tiles
    (1537, 3000, 3200),   # gated backward, NT and NN: pairs, the last waves stream-K; TN: waves, one warp
    (257, 1544, 2050),    # NN: stream-K on single CTAs
    (1537, 1032, 3200),   # NN: stream-K on pairs, fewer tiles than walkers
    (1537, 3000, 1408),   # NN: pairs, the last waves stream-K; NT: waves of tiles, one warp
    (1030, 1032, 2560),   # NT: stream-K on single CTAs; gated: one wave of pairs
    (2600, 1032, 520),    # TN: stream-K on single CTAs, fewer tiles than walkers; NT and NN: one wave of pairs
    (40, 1544, 3200),     # TN: single CTAs, the last waves stream-K
    (2600, 1000, 2560),   # TN: pairs, the last waves stream-K
]


@pytest.mark.parametrize("size", LARGE, ids=str)
@pytest.mark.parametrize("act,dt", [("silu", "bf16"), ("gelu", "f16")])
def test_large_blocks(size, act, dt):
    check_block(size, act, dt, repeats=2)


# The same for the updates: X X^T (NT) or X^T X (TN) and B on the tiles on and
# above the diagonal, mirrored; a X + B X (diagonal by rows) or X B (by columns).
UPDATES = [
    (400, 6000),          # by rows: one wave of pairs
    (1000, 6000),         # by rows: pairs, waves of tiles, two warps
    (1100, 4100),         # X X^T: stream-K on single CTAs; by rows: waves of those
    (1800, 6000),         # X X^T: stream-K on pairs; by rows: pairs, waves, one warp
    (2100, 2300),         # X X^T and B: symmetric on pairs
    (2100, 4100),         # by rows: pairs, the last waves stream-K
]


@pytest.mark.parametrize("shape", UPDATES + [s[::-1] for s in UPDATES], ids=str)
def test_large_updates(shape):
    check_update(*shape, repeats=2)


def test_a_batch_of_updates_on_pairs():
    g = torch.stack([gradient(700, 2304, seed=i) for i in range(6)]).cuda()
    got = sg.orthogonalize(g)
    for i in range(6):
        exact, model = iterate(g[i]), iterate(g[i], rounded=True)
        off = float((got[i].double() - exact).norm() / exact.norm())
        assert off <= 1.5 * float((model - exact).norm() / exact.norm()) + 2.0 ** -9, i
    assert torch.equal(sg.orthogonalize(g), got)
