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
