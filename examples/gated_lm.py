"""A small next-token model trained and sampled with this package's kernels.

    python examples/gated_lm.py [--steps 60] [--tokens 2048] [--vocab 512]
        [--width 256] [--inner 704]

One gated feed-forward block between an embedding and a head, on synthetic
text whose next token is a fixed function of the last one nine times in ten.
A step is a forward pass (gated_ffn, matmul_nt), the loss and its gradient
(token_logprobs, token_logprobs_backward), the backward pass (matmul_nn,
matmul_nt, gated_ffn_backward) and an orthogonalised momentum update of the
weights (orthogonalize).  Afterwards the model continues a sequence token by
token and prints each token's best alternatives.  PyTorch does the rest: the
embedding's gather and scatter, sums, and the momentum.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import software_pipelined_tiled_gemm_gb300 as sg  # noqa: E402


class GatedLM:
    """embedding -> x + block(x) -> head; fp32 weights, bf16 copies in use."""

    def __init__(self, vocab, width, inner, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def init(rows, cols):
            return torch.randn(rows, cols, generator=g, device="cuda") * cols ** -0.5
        self.master = {"embedding": init(vocab, width) * width ** 0.5, "w_in": init(2 * inner, width),
                       "w_out": init(width, inner), "head": init(vocab, width)}
        self.momentum = {k: torch.zeros_like(v) for k, v in self.master.items()}
        self.refresh()

    def refresh(self):
        self.w = {k: v.to(torch.bfloat16) for k, v in self.master.items()}

    def forward(self, tokens, save=False):
        """Logits in fp32 and, with save, what the backward pass needs."""
        x = self.w["embedding"][tokens]
        if save:
            y, kept = sg.gated_ffn(x, self.w["w_in"], self.w["w_out"], act="silu", save=True)
        else:
            y, kept = sg.gated_ffn(x, self.w["w_in"], self.w["w_out"], act="silu"), None
        out = x + y
        logits = sg.matmul_nt(out, self.w["head"], out_dtype=torch.float32)
        return logits, (tokens, x, out, kept)

    def backward(self, d_logits, saved):
        tokens, x, out, kept = saved
        d = d_logits.to(torch.bfloat16)
        d_out = sg.matmul_nn(d, self.w["head"])
        d_head = sg.matmul_nt(d.t().contiguous(), out.t().contiguous(), out_dtype=torch.float32)
        dx, dw_in, dw_out = sg.gated_ffn_backward(d_out, x, self.w["w_in"], self.w["w_out"], kept)
        d_embedding = torch.zeros_like(self.master["embedding"])
        d_embedding.index_add_(0, tokens, (dx + d_out).float())
        return {"embedding": d_embedding, "w_in": dw_in, "w_out": dw_out, "head": d_head}

    def update(self, grads, lr, beta=0.9):
        for name, g in grads.items():
            m, w = self.momentum[name], self.master[name]
            m.mul_(beta).add_(g.float(), alpha=1 - beta)
            if name == "embedding":
                w.sub_(m / m.norm(dim=1, keepdim=True).clamp(min=1e-12), alpha=lr)
                continue
            # The two halves of w_in are matrices of their own.
            parts = m.view(2, -1, m.shape[1]) if name == "w_in" else m.unsqueeze(0)
            step = sg.orthogonalize(parts)
            scale = lr * max(1.0, parts.shape[1] / parts.shape[2]) ** 0.5
            w.view(parts.shape).sub_(step.float(), alpha=scale)
        self.refresh()


def text(count, vocab, seed):
    """`count` tokens; each is 5 t + 7 of the last one t, or one time in ten any."""
    g = torch.Generator().manual_seed(seed)
    noise = torch.rand(count, generator=g) < 0.1
    any_ = torch.randint(0, vocab, (count,), generator=g).tolist()
    out, t = [], 1
    for i in range(count):
        t = any_[i] if noise[i] else (5 * t + 7) % vocab
        out.append(t)
    return torch.tensor(out, device="cuda")


def train(model, steps, tokens, vocab, lr=0.05, log=print):
    losses = []
    for step in range(steps):
        data = text(tokens + 1, vocab, seed=step)
        logits, saved = model.forward(data[:-1], save=True)
        r = sg.token_logprobs(logits, data[1:])
        weight = torch.full_like(r.logprobs, -1.0 / tokens)     # the loss is -mean log p
        d_logits = sg.token_logprobs_backward(logits, data[1:], r, weight, out=logits)
        model.update(model.backward(d_logits, saved), lr * (1 - step / steps))
        losses.append(r.logprobs)
        if log and (step % 10 == 0 or step + 1 == steps):
            log("step %3d  loss %.4f  entropy %.4f" % (step, -float(r.logprobs.mean()), float(r.entropy.mean())))
    return [-float(x.mean()) for x in losses]


def generate(model, start, count, top_k=3, log=print):
    """Continue from one token greedily, one token a call."""
    tokens = [start]
    for _ in range(count):
        logits, _ = model.forward(torch.tensor(tokens[-1:], device="cuda"))
        r = sg.token_logprobs(logits, top_k=top_k)
        ids, lps = r.top_ids[0].tolist(), r.top_logprobs[0].tolist()
        if log:
            log("%4d -> " % tokens[-1] + "  ".join("%d (%.3f)" % (i, math.exp(p)) for i, p in zip(ids, lps)))
        tokens.append(ids[0])
    return tokens


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--vocab", type=int, default=512)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--inner", type=int, default=704)
    args = ap.parse_args(argv)
    model = GatedLM(args.vocab, args.width, args.inner)
    losses = train(model, args.steps, args.tokens, args.vocab)
    generate(model, 1, 8)
    sg.check_operators()
    return losses


if __name__ == "__main__":
    main()
