"""A copy that never lands: the operators' device waits run out after their
limit, the kernels finish, the status word says so, and the next call on the
same handle is right.  Nothing faults or hangs: the hook only leaves one copy
out (gemm_ops_configure)."""
from __future__ import annotations

import time

import pytest
import torch

import software_pipelined_tiled_gemm_gb300 as sg
from software_pipelined_tiled_gemm_gb300 import operators

pytestmark = pytest.mark.gpu


def _tensors(m, d, i):
    g = torch.Generator().manual_seed(m)
    return [torch.randn(*s, generator=g).mul(s[-1] ** -0.5).bfloat16().cuda()
            for s in ((m, d), (2 * i, d), (d, i))]


def _cases():
    one = _tensors(1, 256, 512)            # shared K of few tiles
    mid = _tensors(200, 256, 320)          # single CTAs, clusters of K shares
    big = _tensors(1500, 1024, 4096)       # CTA pairs
    grad = torch.randn(300, 200, generator=torch.Generator().manual_seed(1)).cuda()
    rows = torch.randn(700, 9000, generator=torch.Generator().manual_seed(2)).cuda()
    row = torch.randn(1, 70000, generator=torch.Generator().manual_seed(3)).cuda()
    return [("ffn %d" % t[0].shape[0], lambda t=t: sg.gated_ffn(*t)) for t in (one, mid, big)] + [
        ("orthogonalize", lambda: sg.orthogonalize(grad)),
        ("logprobs", lambda: sg.token_logprobs(rows, None, top_k=4).lse),
        ("logprobs shared row", lambda: sg.token_logprobs(row, None, top_k=4).lse)]


@pytest.mark.parametrize("which", range(6))
def test_timeout_is_reported_and_the_next_call_is_right(which):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dev = torch.device("cuda", 0)
    name, call = _cases()[which]
    want = call()
    sg.check_operators()
    try:
        operators._configure(dev, timeout_ns=20_000_000, debug_fault=1)
        t0 = time.perf_counter()
        call()
        with pytest.raises(sg.GemmError) as e:
            sg.check_operators()
        assert e.value.status == sg.GEMM_ERR_TIMEOUT, name
        assert time.perf_counter() - t0 < 20.0
    finally:
        operators._configure(dev)
    got = call()
    sg.check_operators()
    assert torch.equal(got, want), name


def test_refusals():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dev = torch.device("cuda", 0)
    for kw in (dict(timeout_ns=-1), dict(debug_fault=2), dict(debug_fault=-1)):
        with pytest.raises(sg.GemmError):
            operators._configure(dev, **kw)
