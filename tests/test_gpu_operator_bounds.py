"""The operators in the bounds-checked build.

Its block products and on-chip updates check tile, K slice, copy coordinates,
ring slot, stored block, workspace slot and shared-memory layout before each
use (the passes over weights for few tokens, the log probabilities and the
copy and norm kernels have no such checks).  A child process that loads that
build runs every schedule; none of the checks fires, and the results are those
of the normal build bit for bit.
"""
from __future__ import annotations

import json
import os
import subprocess
import sys
import textwrap

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

_CODE = """
    import json
    import torch
    import software_pipelined_tiled_gemm_gb300 as sg
    from tests.test_gpu_gated_ffn import inputs, run_all
    from tests.test_gpu_operator_schedules import CLUSTER, LARGE, UPDATES
    from tests.test_gpu_orthogonalize import gradient

    def digest(t):
        # Two sums of the bits, one of them weighted by place: whole numbers, so in any order.
        w = t.contiguous().view(torch.int16).reshape(-1).long()
        place = torch.arange(w.numel(), device=w.device) % 65521
        return [int(w.sum()), int((w * place).sum())]

    out = {"checked": sg.gemm_bounds_checked(), "digests": []}
    for size in CLUSTER + LARGE + [(200, 512, 704), (33, 67, 101)]:
        got = run_all(*(t.cuda() for t in inputs(*size, "bf16", seed=1)), "silu")
        out["digests"] += [digest(got[k]) for k in sorted(got)]
    for m, n in UPDATES + [(260, 1200), (64, 64), (256, 640), (200, 300), (128, 4097)]:
        for shape in ((m, n), (n, m)):
            out["digests"].append(digest(sg.orthogonalize(gradient(*shape, seed=2).cuda())))
    sg.check_operators()
    print(json.dumps(out))
"""


def _child(checked):
    env = dict(os.environ, SPGEMM_BOUNDS_CHECKS="1" if checked else "0")
    out = subprocess.run([sys.executable, "-c", textwrap.dedent(_CODE)], cwd=ROOT, env=env, capture_output=True,
                         text=True, timeout=600)
    assert out.returncode == 0, out.stderr[-4000:]
    return json.loads(out.stdout.strip().splitlines()[-1])


@pytest.mark.gpu
def test_no_check_fires_and_the_results_are_the_same():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    checked, normal = _child(True), _child(False)
    assert checked["checked"] == 1 and normal["checked"] == 0
    assert checked["digests"] == normal["digests"]
