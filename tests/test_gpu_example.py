"""The example model learns its synthetic text through the package's kernels."""
from __future__ import annotations

import math
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.gpu
def test_training_and_generation():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_lm
    import software_pipelined_tiled_gemm_gb300 as sg
    vocab = 512
    model = gated_lm.GatedLM(vocab, 256, 704)
    losses = gated_lm.train(model, steps=60, tokens=2048, vocab=vocab, log=None)
    sg.check_operators()
    # From about a uniform guess, ln 512, to well under half of it (the text's
    # own entropy is near 0.95).
    assert 0.8 * math.log(vocab) < losses[0] < 2 * math.log(vocab)
    assert losses[-1] < 0.5 * math.log(vocab)
    tokens = gated_lm.generate(model, 1, 8, log=None)
    rule = sum(b == (5 * a + 7) % vocab for a, b in zip(tokens, tokens[1:]))
    assert rule >= 6


@pytest.mark.gpu
def test_gradients_of_the_whole_model_against_differences():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_lm
    import software_pipelined_tiled_gemm_gb300 as sg
    model = gated_lm.GatedLM(64, 48, 40, seed=3)
    data = gated_lm.text(129, 64, seed=1)

    def loss(w):
        x = w["embedding"][data[:-1]]
        gu = x @ w["w_in"].T
        out = x + (gu[:, :40] * torch.sigmoid(gu[:, :40]) * gu[:, 40:]) @ w["w_out"].T
        return -torch.log_softmax(out @ w["head"].T, 1).gather(1, data[1:, None]).mean()

    logits, saved = model.forward(data[:-1], save=True)
    r = sg.token_logprobs(logits, data[1:])
    d = sg.token_logprobs_backward(logits, data[1:], r, torch.full_like(r.logprobs, -1.0 / 128))
    grads = model.backward(d, saved)
    point = {k: v.double() for k, v in model.w.items()}
    assert abs(float(loss(point)) + float(r.logprobs.double().mean())) < 2e-2   # bf16 y and x + y
    for name in grads:
        v = torch.randn(point[name].shape, dtype=torch.float64, device="cuda",
                        generator=torch.Generator(device="cuda").manual_seed(5))
        hi, lo = dict(point), dict(point)
        hi[name], lo[name] = point[name] + 1e-5 * v, point[name] - 1e-5 * v
        diff = float(loss(hi) - loss(lo)) / 2e-5
        mine = float((grads[name].double() * v).sum())
        # bf16 roundings of y, x + y, d_logits, d_out and the gradient, each 2^-8 of
        # vectors no longer than the gradient's contributions, in random directions
        assert abs(mine - diff) < 5 * 2.0 ** -8 * float(grads[name].double().norm()) * 3, (name, mine, diff)
