"""A small next-token model with a layer of experts, trained and sampled with this package's kernels.

    python examples/expert_lm.py [--steps 60] [--tokens 2048] [--vocab 512]
        [--width 256] [--inner 352] [--experts 8]

embedding -> x + p expert(norm(x)) -> head, on the text of gated_lm.py.  Each
token goes to the expert that a router likes best, weighted by the router's
probability p for it.  A step is a forward pass (layer_norm, matmul_nt for the
router and the head, grouped_matmul for the experts' two products), the loss
and its gradient (token_logprobs, token_logprobs_backward), the backward pass
(matmul_nn, matmul_nt, grouped_matmul_backward, layer_norm_backward), an
orthogonalised momentum update of the experts' matrices (orthogonalize) and an
AdamW step of everything else (adamw, states in 8 bits).  PyTorch does the rest:
gathers, scatters, the activation between the products, the choice of experts.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
for path in (HERE, os.path.dirname(HERE)):
    if path not in sys.path:
        sys.path.insert(0, path)

import software_pipelined_tiled_gemm_gb300 as sg  # noqa: E402
from gated_lm import text  # noqa: E402

EXPERT = ("w_in", "w_out")   # matrices, one of a kind for each expert


class ExpertLM:
    """fp32 weights with bf16 copies in use (the norm's vectors are used as they are)."""

    def __init__(self, vocab, width, inner, experts, seed=0, bits=8):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def init(*shape):
            return torch.randn(*shape, generator=g, device="cuda") * shape[-1] ** -0.5
        self.experts, self.inner = experts, inner
        self.master = {"embedding": init(vocab, width) * width ** 0.5, "norm_w": torch.ones(width, device="cuda"),
                       "norm_b": torch.zeros(width, device="cuda"), "router": init(experts, width),
                       "w_in": init(experts, 2 * inner, width), "w_out": init(experts, width, inner),
                       "head": init(vocab, width)}
        self.w = {k: v if k.startswith("norm") else v.to(torch.bfloat16) for k, v in self.master.items()}
        self.momentum = {k: torch.zeros_like(self.master[k]) for k in EXPERT}
        self.others = [k for k in self.master if k not in EXPERT]
        self.state = sg.adamw_state([self.master[k] for k in self.others], bits=bits)

    def forward(self, tokens):
        """Logits in fp32, and what the backward pass needs."""
        w, s = self.w, {"tokens": tokens}
        s["x"] = w["embedding"][tokens]
        s["h"], s["kept"] = sg.layer_norm(s["x"], w["norm_w"], w["norm_b"], save=True)
        s["p"] = torch.softmax(sg.matmul_nt(s["h"], w["router"], out_dtype=torch.float32), 1)
        s["best"] = s["p"].argmax(1)
        s["order"] = torch.argsort(s["best"], stable=True)      # rows by expert
        counts = torch.zeros(self.experts + 1, dtype=torch.int64, device="cuda")
        counts.index_add_(0, s["best"] + 1, torch.ones_like(s["best"]))
        s["offsets"] = counts.cumsum(0)
        s["rows"] = s["h"][s["order"]]
        gu = sg.grouped_matmul(s["rows"], w["w_in"], s["offsets"]).float()
        s["gate"], s["up"] = gu[:, :self.inner], gu[:, self.inner:]
        s["inner"] = (torch.nn.functional.silu(s["gate"]) * s["up"]).to(torch.bfloat16)
        s["y"] = sg.grouped_matmul(s["inner"], w["w_out"], s["offsets"])
        s["weight"] = s["p"].gather(1, s["best"][:, None])[s["order"]]
        out = s["x"].float()
        out[s["order"]] += s["weight"] * s["y"].float()
        s["out"] = out.to(torch.bfloat16)
        return sg.matmul_nt(s["out"], w["head"], out_dtype=torch.float32), s

    def backward(self, d_logits, s):
        w, order = self.w, s["order"]
        d = d_logits.to(torch.bfloat16)
        d_out = sg.matmul_nn(d, w["head"])
        grads = {"head": sg.matmul_nt(d.t().contiguous(), s["out"].t().contiguous(), out_dtype=torch.float32)}
        d_rows = d_out[order].float()
        d_y = (s["weight"] * d_rows).to(torch.bfloat16)
        d_inner, grads["w_out"] = sg.grouped_matmul_backward(d_y, s["inner"], w["w_out"], s["offsets"])
        sig = torch.sigmoid(s["gate"])
        d_gu = torch.cat([d_inner * s["up"] * sig * (1 + s["gate"] * (1 - sig)), d_inner * s["gate"] * sig], 1)
        d_h_rows, grads["w_in"] = sg.grouped_matmul_backward(d_gu.to(torch.bfloat16), s["rows"], w["w_in"], s["offsets"])
        d_h = torch.empty_like(s["h"], dtype=torch.float32)
        d_h[order] = d_h_rows.float()
        # The router: d p_best = <d_out, y>, through the softmax.
        d_best = torch.empty(len(order), 1, device="cuda")
        d_best[order] = (d_rows * s["y"].float()).sum(1, keepdim=True)
        best = torch.nn.functional.one_hot(s["best"], self.experts)
        d_r = (d_best * s["p"].gather(1, s["best"][:, None]) * (best - s["p"])).to(torch.bfloat16)
        grads["router"] = sg.matmul_nt(d_r.t().contiguous(), s["h"].t().contiguous(), out_dtype=torch.float32)
        d_h = (d_h + d_r.float() @ w["router"].float()).to(torch.bfloat16)
        d_x, grads["norm_w"], grads["norm_b"] = sg.layer_norm_backward(d_h, s["x"], w["norm_w"], s["kept"])
        grads["embedding"] = torch.zeros_like(self.master["embedding"]).index_add_(0, s["tokens"], (d_x + d_out).float())
        return grads

    def update(self, grads, lr, beta=0.9):
        for name in EXPERT:
            m, w = self.momentum[name], self.master[name]
            m.mul_(beta).add_(grads[name].float(), alpha=1 - beta)
            # The two halves of an expert's w_in are matrices of their own.
            parts = m.view(-1, self.inner, m.shape[2]) if name == "w_in" else m
            step = sg.orthogonalize(parts)
            w.view(parts.shape).sub_(step.float(), alpha=lr * max(1.0, parts.shape[1] / parts.shape[2]) ** 0.5)
            self.w[name].copy_(w)
        names = self.others
        sg.adamw([self.master[k] for k in names], [grads[k] for k in names], self.state, lr=0.2 * lr,
                 weight_decay=[0.0 if k.startswith("norm") else 0.01 for k in names],
                 copies=[None if k.startswith("norm") else self.w[k] for k in names])


def train(model, steps, tokens, vocab, lr=0.05, log=print):
    losses = []
    for step in range(steps):
        data = text(tokens + 1, vocab, seed=step)
        logits, saved = model.forward(data[:-1])
        r = sg.token_logprobs(logits, data[1:])
        weight = torch.full_like(r.logprobs, -1.0 / tokens)     # the loss is -mean log p
        d_logits = sg.token_logprobs_backward(logits, data[1:], r, weight, out=logits)
        model.update(model.backward(d_logits, saved), lr * (1 - step / steps))
        losses.append(r.logprobs)
        if log and (step % 10 == 0 or step + 1 == steps):
            counts = torch.diff(saved["offsets"]).tolist()
            log("step %3d  loss %.4f  tokens of each expert %s" % (step, -float(r.logprobs.mean()), counts))
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
    ap.add_argument("--inner", type=int, default=352)
    ap.add_argument("--experts", type=int, default=8)
    args = ap.parse_args(argv)
    model = ExpertLM(args.vocab, args.width, args.inner, args.experts)
    losses = train(model, args.steps, args.tokens, args.vocab)
    generate(model, 1, 8)
    sg.check_operators()
    return losses


if __name__ == "__main__":
    main()
