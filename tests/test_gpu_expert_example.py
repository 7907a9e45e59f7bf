"""The example with a layer of experts: it runs through the package's kernels,
and its gradients are those of its formula."""
from __future__ import annotations

import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("bits", [8, 32])
def test_training_and_generation_run(bits):
    import expert_lm
    import software_pipelined_tiled_gemm_gb300 as sg
    model = expert_lm.ExpertLM(200, 96, 40, 5, bits=bits)
    before = {k: v.clone() for k, v in model.w.items()}
    losses = expert_lm.train(model, steps=6, tokens=300, vocab=200, log=None)
    assert all(0 < x < 100 for x in losses)
    assert len(expert_lm.generate(model, 1, 4, log=None)) == 5
    sg.check_operators()
    assert int(model.state.step) == 6
    for k, v in model.w.items():
        assert torch.isfinite(v).all() and not torch.equal(v, before[k]), k
        if not k.startswith("norm"):
            assert torch.equal(v, model.master[k].to(torch.bfloat16)), k


def test_gradients_of_the_whole_model_against_differences():
    import expert_lm
    import software_pipelined_tiled_gemm_gb300 as sg
    model = expert_lm.ExpertLM(64, 48, 40, 4, seed=3)
    model.w["norm_w"].mul_(1.1)
    data = expert_lm.text(129, 64, seed=1)
    logits, s = model.forward(data[:-1])
    best = s["best"]      # (far from a tie next to the differences' step)

    def loss(w):
        x = w["embedding"][data[:-1]]
        h = torch.nn.functional.layer_norm(x, (48,), w["norm_w"], w["norm_b"])
        p = torch.softmax(h @ w["router"].T, 1).gather(1, best[:, None])
        gu = torch.einsum("td,tid->ti", h, w["w_in"][best])
        y = torch.einsum("ti,tdi->td", torch.nn.functional.silu(gu[:, :40]) * gu[:, 40:], w["w_out"][best])
        return -torch.log_softmax((x + p * y) @ w["head"].T, 1).gather(1, data[1:, None]).mean()

    r = sg.token_logprobs(logits, data[1:])
    d = sg.token_logprobs_backward(logits, data[1:], r, torch.full_like(r.logprobs, -1.0 / 128))
    grads = model.backward(d, s)
    point = {k: v.double() for k, v in model.w.items()}
    assert abs(float(loss(point)) + float(r.logprobs.double().mean())) < 2e-2   # bf16 h, y and x + p y
    for name in grads:
        v = torch.randn(point[name].shape, dtype=torch.float64, device="cuda",
                        generator=torch.Generator(device="cuda").manual_seed(5))
        hi, lo = dict(point), dict(point)
        hi[name], lo[name] = point[name] + 1e-5 * v, point[name] - 1e-5 * v
        diff = float(loss(hi) - loss(lo)) / 2e-5
        mine = float((grads[name].double() * v).sum())
        # bf16 roundings of h, the products, y, x + p y, d_logits, d_out, d_y, d_gu, d_h and the
        # gradient, each 2^-8 of vectors no longer than the gradient's contributions, in random directions
        assert abs(mine - diff) < 10 * 2.0 ** -8 * float(grads[name].double().norm()) * 3, (name, mine, diff)


def test_a_captured_training_step_repeats():
    """The operators of a step, captured together and replayed: gradients and AdamW update as eagerly."""
    import expert_lm
    import software_pipelined_tiled_gemm_gb300 as sg
    data = expert_lm.text(257, 128, seed=2)

    def step(model):
        logits, s = model.forward(data[:-1])
        r = sg.token_logprobs(logits, data[1:])
        grads = model.backward(sg.token_logprobs_backward(logits, data[1:], r, torch.full_like(r.logprobs, -1.0 / 256)), s)
        model.update(grads, 0.02)
        return grads

    a, b = (expert_lm.ExpertLM(128, 64, 72, 4, seed=6) for _ in range(2))
    for model in (a, b):
        step(model)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = step(a)
    for _ in range(3):
        graph.replay()
        eager = step(b)
    torch.cuda.synchronize()
    sg.check_operators()
    assert int(a.state.step) == int(b.state.step) == 4
    # (The embedding's gradient is summed by PyTorch's atomics, in no fixed order.)
    for k in eager:
        if k == "embedding":
            assert torch.allclose(held[k], eager[k], rtol=1e-4, atol=1e-6)
