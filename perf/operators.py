"""The operators around the GEMM that a model's layers, loss and optimiser need.

Three operators, each with a plain form in elementary torch operations and
the call a user makes of this framework:

gated feed-forward block    y = (act(x Wg^T) * (x Wu^T)) Wo^T, with w_in = [Wg; Wu] stored
                            as one (2 I, D) matrix and w_out = Wo (D, I); for training also
                            the gradients of x, w_in and w_out
orthogonalised update       the matrix sign of a gradient by Newton-Schulz products:
                            X = G / |G|_F, then X <- a X + (b A + c A^2) X with A = X X^T
token log probabilities     of given tokens under rows of logits, with the entropy and the
                            best alternatives of each row; for training also the gradient

A case is a dict of plain values; prepare() makes its inputs on the GPU from a
seed, run() makes one pass, exact() gives the same outputs from the definition
in 64 bits.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}
_COEFFS = (3.4445, -4.7750, 2.0315)
_STEPS = 5

# ------------------------------------------------------------------ cases --


def listed():
    return [
        # One token through a layer while serving: latency and the weights' bytes.
        {"name": "ffn token", "op": "ffn", "m": 1, "d": 4096, "i": 16384, "act": "silu", "type": "bf16"},
        # A batch of sequences decoding together.
        {"name": "ffn batch 64", "op": "ffn", "m": 64, "d": 8192, "i": 8192, "act": "silu", "type": "f16"},
        # A prompt of odd length through a layer whose sizes fit no tile and no 16-byte row.
        {"name": "ffn ragged", "op": "ffn", "m": 1023, "d": 1531, "i": 4097, "act": "gelu", "type": "bf16"},
        # A long prompt.
        {"name": "ffn prompt", "op": "ffn", "m": 8192, "d": 4096, "i": 16384, "act": "silu", "type": "bf16"},
        # A training step of a small layer, forward and backward.
        {"name": "ffn train small", "op": "ffn_train", "m": 640, "d": 512, "i": 1408, "act": "gelu", "type": "f16"},
        # A training step of a large layer.
        {"name": "ffn train", "op": "ffn_train", "m": 8192, "d": 4096, "i": 16384, "act": "silu", "type": "bf16"},
        # A stack of small weights (one for each head, or the experts of a small model).
        {"name": "orthogonal stack", "op": "orthogonal", "b": 8, "m": 256, "n": 640, "type": "f32"},
        # A tall weight with odd sides.
        {"name": "orthogonal tall", "op": "orthogonal", "b": 1, "m": 4097, "n": 1000, "type": "bf16"},
        # One large weight of a layer.
        {"name": "orthogonal large", "op": "orthogonal", "b": 1, "m": 4096, "n": 16384, "type": "f32"},
        # The next token's distribution while serving: its log probability and 20 alternatives.
        {"name": "logprobs token", "op": "logprobs", "t": 1, "v": 131072, "k": 20, "type": "bf16", "masked": False},
        # Scoring a prompt under a vocabulary that ends in masked padding, five alternatives a token.
        {"name": "logprobs prompt", "op": "logprobs", "t": 4096, "v": 128257, "k": 5, "type": "f32", "masked": True},
        # The loss of a training step, forward and backward, with an entropy bonus.
        {"name": "logprobs train", "op": "logprobs_train", "t": 8192, "v": 65536, "k": 0, "type": "bf16", "masked": False},
    ]


def _between(rng, lo, hi):
    """A size spread over the logarithm of [lo, hi], odd ones among them."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ffn", "ffn", "ffn_train", "orthogonal", "logprobs", "logprobs_train"])
    while True:
        if op in ("ffn", "ffn_train"):
            # Widths of a layer are multiples of 8 in most models, and anything in the rest.
            step = rng.choice([64, 64, 8, 1])
            case = {"op": op, "m": _between(rng, 1, 8192),
                    "d": max(step, _between(rng, 256, 8192) // step * step),
                    "i": max(step, _between(rng, 512, 16384) // step * step),
                    "act": rng.choice(["silu", "silu", "gelu", "relu"]), "type": rng.choice(["bf16", "f16"])}
        elif op == "orthogonal":
            step = rng.choice([64, 8, 1])
            case = {"op": op, "b": rng.choice([1, 1, _between(rng, 1, 16)]),
                    "m": max(step, _between(rng, 64, 8192) // step * step),
                    "n": max(step, _between(rng, 64, 8192) // step * step),
                    "type": rng.choice(["f32", "bf16", "f16"])}
        else:
            case = {"op": op, "t": _between(rng, 1, 8192), "v": _between(rng, 500, 200000),
                    "k": 0 if op == "logprobs_train" else rng.choice([0, 1, 5, 20, 50]),
                    "type": rng.choice(["bf16", "bf16", "f32", "f16"]), "masked": rng.random() < 0.4}
        w = work(case)
        # Not above the largest listed case of its operator.
        if w["flops"] <= {"ffn": 3.3e12, "ffn_train": 9.9e12, "orthogonal": 4.5e12}.get(op, 1e99) and (
                "logprobs" not in op or w["bytes"] <= 2.1e9):
            return case


def work(case):
    e = _SIZE[case["type"]]
    if case["op"] == "ffn":
        m, d, i = case["m"], case["d"], case["i"]
        return {"bytes": e * (2 * m * d + 3 * d * i), "flops": 6 * m * d * i}
    if case["op"] == "ffn_train":
        m, d, i = case["m"], case["d"], case["i"]
        return {"bytes": e * (4 * m * d + 6 * d * i), "flops": 18 * m * d * i}
    if case["op"] == "orthogonal":
        # With m <= n: X X^T and A^2 are symmetric, so half of each product is enough.
        b, m, n = case["b"], min(case["m"], case["n"]), max(case["m"], case["n"])
        return {"bytes": b * m * n * (e + 2), "flops": _STEPS * b * (3 * m * m * n + m * m * m)}
    t, v, k = case["t"], case["v"], case["k"]
    forward = t * v * e + t * (8 + 12 + 12 * k)
    if case["op"] == "logprobs":
        return {"bytes": forward, "flops": 6 * t * v}
    return {"bytes": forward + t * (8 + 16) + 2 * t * v * e, "flops": 12 * t * v}


# ----------------------------------------------------------------- inputs --


def prepare(case, seed):
    dt = _TYPES[case["type"]]
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale)

    s = {"case": dict(case)}
    if case["op"] in ("ffn", "ffn_train"):
        m, d, i = case["m"], case["d"], case["i"]
        # A normalised hidden state with some channels larger than the rest, and weights
        # that keep its scale.
        s["x"] = (normal(m, d) * (1.0 + 2.0 * (torch.rand(d, generator=g, device="cuda") > 0.98))).to(dt)
        s["w_in"] = normal(2 * i, d, scale=d ** -0.5).to(dt)
        s["w_out"] = normal(d, i, scale=i ** -0.5).to(dt)
        if case["op"] == "ffn_train":
            s["dy"] = normal(m, d, scale=0.1).to(dt)
    elif case["op"] == "orthogonal":
        # A momentum of gradients: a few strong directions over noise, at a small scale.
        b, m, n = case["b"], case["m"], case["n"]
        r = max(1, min(m, n) // 16)
        low = torch.bmm(normal(b, m, r), normal(b, r, n)) * (2.0 / r ** 0.5)
        s["g"] = ((low + normal(b, m, n)) * 1e-3).to(dt)
        if b == 1:
            s["g"] = s["g"][0]
    else:
        t, v = case["t"], case["v"]
        # Rows of different sharpness, from nearly flat to nearly decided.
        x = normal(t, v) * (0.5 + 3.0 * torch.rand(t, 1, generator=g, device="cuda"))
        if case["masked"]:
            # The vocabulary's padding, and the tokens that a grammar forbids in some rows.
            x[:, v - v // 100:] = -math.inf
            rows = torch.rand(t, 1, generator=g, device="cuda") < 0.25
            x.masked_fill_(rows & (torch.rand(1, v, generator=g, device="cuda") < 0.9), -math.inf)
        s["logits"] = x.to(dt)
        del x
        s["tokens"] = torch.randint(0, max(1, v - v // 100), (t,), generator=g, device="cuda")
        if t > 1:
            s["tokens"][::17] = -100  # prompt positions that no loss is taken of
        if case["op"] == "logprobs_train":
            # The gradient of a mean over tokens, under the loss scale that fp16 gradients need.
            scale = (32768.0 if case["type"] == "f16" else 1.0) / t
            s["d_logprobs"] = -torch.rand(t, generator=g, device="cuda") * scale
            s["d_entropy"] = normal(t, scale=0.01 * scale)
    return s


# ------------------------------------------------------------ plain forms --


def _act(name, g):
    """The activation and its derivative."""
    if name == "relu":
        return torch.clamp(g, min=0.0), (g > 0).to(g.dtype)
    if name == "silu":
        p = 1.0 / (1.0 + torch.exp(-g))
        return g * p, p * (1.0 + g * (1.0 - p))
    c = 0.7978845608
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g)


def _plain_ffn(s):
    c, dt = s["case"], s["x"].dtype
    x, w_in, w_out = s["x"].float(), s["w_in"].float(), s["w_out"].float()
    i = c["i"]
    gu = x @ w_in.t()
    gate, up = gu[:, :i], gu[:, i:]
    a, da = _act(c["act"], gate)
    h = a * up
    y = (h @ w_out.t()).to(dt)
    if c["op"] == "ffn":
        return {"y": y}
    dy = s["dy"].float()
    dh = dy @ w_out
    dgu = torch.cat([dh * up * da, dh * a], 1)
    return {"y": y, "dx": (dgu @ w_in).to(dt), "dw_in": (dgu.t() @ x).to(dt), "dw_out": (dy.t() @ h).to(dt)}


def _plain_orthogonal(s):
    g = s["g"].float()
    tall = g.shape[-2] > g.shape[-1]
    x = g.transpose(-1, -2) if tall else g
    x = x / torch.clamp((x * x).sum((-2, -1), keepdim=True).sqrt(), min=1e-7)
    a, b, c = _COEFFS
    for _ in range(_STEPS):
        p = x @ x.transpose(-1, -2)
        x = a * x + (b * p + c * (p @ p)) @ x
    return {"update": (x.transpose(-1, -2) if tall else x).to(torch.bfloat16).contiguous()}


def _plain_logprobs(s):
    c, tokens = s["case"], s["tokens"]
    x = s["logits"].float()
    top = x.amax(1, keepdim=True)
    top = torch.where(torch.isinf(top) & (top < 0), torch.zeros_like(top), top)
    lse = top + torch.exp(x - top).sum(1, keepdim=True).log()
    lp = torch.where(torch.isinf(x) & (x < 0), x, x - lse)
    p = torch.exp(lp)
    plp = torch.where(p > 0, p * lp, torch.zeros_like(lp))
    entropy = -plp.sum(1)
    picked = lp.gather(1, tokens.clamp(min=0).unsqueeze(1))[:, 0]
    out = {"logprobs": torch.where(tokens < 0, torch.zeros_like(picked), picked), "entropy": entropy}
    if c["k"]:
        # Best first, equal ones by the lowest index: one whole number orders both.
        bits = (x + 0.0).view(torch.int32)
        order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).to(torch.int64)
        place = (1 << 20) - 1 - torch.arange(x.shape[1], device=x.device)
        keys = torch.topk(order * (1 << 20) + place, c["k"], dim=1).values
        ids = (1 << 20) - 1 - (keys & ((1 << 20) - 1))
        out["top_ids"], out["top_logprobs"] = ids, lp.gather(1, ids)
    if c["op"] == "logprobs_train":
        dl = s["d_logprobs"].masked_fill(tokens < 0, 0.0).unsqueeze(1)
        d = -dl * p - s["d_entropy"].unsqueeze(1) * (plp + p * entropy.unsqueeze(1))
        d.scatter_add_(1, tokens.clamp(min=0).unsqueeze(1), dl)
        out["d_logits"] = d.to(s["logits"].dtype)
    return out


# -------------------------------------------------------------- the calls --


def _own_ffn(s):
    import software_pipelined_tiled_gemm_gb300 as sg
    c = s["case"]
    if c["op"] == "ffn":
        return {"y": sg.gated_ffn(s["x"], s["w_in"], s["w_out"], act=c["act"])}
    y, saved = sg.gated_ffn(s["x"], s["w_in"], s["w_out"], act=c["act"], save=True)
    dx, dw_in, dw_out = sg.gated_ffn_backward(s["dy"], s["x"], s["w_in"], s["w_out"], saved)
    return {"y": y, "dx": dx, "dw_in": dw_in, "dw_out": dw_out}


def _own_orthogonal(s):
    import software_pipelined_tiled_gemm_gb300 as sg
    return {"update": sg.orthogonalize(s["g"], steps=_STEPS, coeffs=_COEFFS, eps=1e-7)}


def _own_logprobs(s):
    import software_pipelined_tiled_gemm_gb300 as sg
    c = s["case"]
    r = sg.token_logprobs(s["logits"], s["tokens"], top_k=c["k"])
    out = {"logprobs": r.logprobs, "entropy": r.entropy}
    if c["k"]:
        out["top_ids"], out["top_logprobs"] = r.top_ids, r.top_logprobs
    if c["op"] == "logprobs_train":
        out["d_logits"] = sg.token_logprobs_backward(s["logits"], s["tokens"], r, s["d_logprobs"],
                                                     s["d_entropy"])
    return out


def run(state):
    op = state["case"]["op"]
    if op in ("ffn", "ffn_train"):
        return _own_ffn(state) if own else _plain_ffn(state)
    if op == "orthogonal":
        return _own_orthogonal(state) if own else _plain_orthogonal(state)
    return _own_logprobs(state) if own else _plain_logprobs(state)


# ----------------------------------------------------- the 64-bit results --


def exact(case, seed):
    """The same outputs in 64 bits; None above a bounded amount of work."""
    if work(case)["flops"] > 1.2e13:
        return None
    s = prepare(case, seed)
    f = {k: v.double() for k, v in s.items() if torch.is_tensor(v) and v.is_floating_point()}
    if case["op"] in ("ffn", "ffn_train"):
        with torch.enable_grad():
            x, w_in, w_out = (f[k].requires_grad_(case["op"] == "ffn_train") for k in ("x", "w_in", "w_out"))
            gate, up = x @ w_in[:case["i"]].T, x @ w_in[case["i"]:].T
            if case["act"] == "silu":
                a = gate * torch.sigmoid(gate)
            elif case["act"] == "gelu":
                a = torch.nn.functional.gelu(gate, approximate="tanh")
            else:
                a = torch.relu(gate)
            y = (a * up) @ w_out.T
            if case["op"] == "ffn":
                return {"y": y}
            dx, dw_in, dw_out = torch.autograd.grad(y, (x, w_in, w_out), f["dy"])
        return {"y": y.detach(), "dx": dx, "dw_in": dw_in, "dw_out": dw_out}
    if case["op"] == "orthogonal":
        x = f["g"]
        x = x / torch.linalg.matrix_norm(x, keepdim=True).clamp(min=1e-7)
        a, b, c = _COEFFS
        for _ in range(_STEPS):
            if x.shape[-1] < x.shape[-2]:  # X (b P + c P^2) with P = X^T X: the same, on the short side
                p = x.mT @ x
                x = a * x + x @ (b * p + c * p @ p)
            else:
                p = x @ x.mT
                x = a * x + (b * p + c * p @ p) @ x
        return {"update": x}
    tokens, rows = s["tokens"], max(1, (1 << 28) // case["v"])
    got = {"logprobs": [], "entropy": []}
    if case["k"]:
        got["top_logprobs"] = []
    if case["op"] == "logprobs_train":
        got["d_logits"] = []
    for r in range(0, case["t"], rows):
        x, tk = f["logits"][r:r + rows], tokens[r:r + rows]
        lp = torch.log_softmax(x, 1)
        h = torch.special.entr(lp.exp()).sum(1)
        idx = tk.clamp(min=0)[:, None]
        got["logprobs"].append(lp.gather(1, idx)[:, 0].masked_fill(tk < 0, 0.0))
        got["entropy"].append(h)
        if case["k"]:
            got["top_logprobs"].append(lp.topk(case["k"], 1).values)
        if case["op"] == "logprobs_train":
            dl = f["d_logprobs"][r:r + rows].masked_fill(tk < 0, 0.0)[:, None]
            p = lp.exp()
            d = -dl * p + f["d_entropy"][r:r + rows, None] * (torch.special.entr(p) - p * h[:, None])
            got["d_logits"].append(d.scatter_add(1, idx, dl))
    out = {k: torch.cat(v) for k, v in got.items()}
    if case["k"]:
        out["top_ids"] = None
    return out


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(n)) for n in range(6)]:
        print(c, work(c))
