"""The operators that a layer of experts is trained and served with.

Three operators, each with a plain form in elementary torch operations and
the call a user makes of this framework:

products grouped by expert  y_r = W_e x_r for the rows r of group e, groups of consecutive rows
                            of any sizes given by their offsets on the GPU, W (E, N, K); for
                            training also the gradients of x and W
layer norm                  y = (x - mean) / sqrt(var + eps) * weight + bias over a row; for
                            training also the gradients of x, weight and bias
AdamW step                  over many tensors at once, with decoupled decay, a factor for the
                            gradients and 16-bit copies of the weights; its states in 32 bits,
                            or in 8 bits with a scale for each 256 elements

A case is a dict of plain values; prepare() makes its inputs on the GPU from a
seed, run() makes one pass, exact() gives the same outputs from the definition
in 64 bits.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4, None: 0}
_EPS = 1e-5
_BETAS, _ADAM_EPS, _LR, _DECAY = (0.9, 0.999), 1e-8, 1e-3, 0.1
_BLOCK = 256

# ------------------------------------------------------------------ cases --


def listed():
    return [
        # One token while serving, sent to eight of 64 experts: eight weights to read, one row each.
        {"name": "experts token", "op": "experts", "t": 8, "e": 64, "n": 2048, "k": 4096, "skew": 0.0, "spare": 0, "type": "bf16"},
        # A batch of sequences decoding together, eight experts a token: every weight for a few rows.
        {"name": "experts batch", "op": "experts", "t": 512, "e": 64, "n": 4096, "k": 2048, "skew": 0.5, "spare": 0, "type": "bf16"},
        # A prompt through a layer of few experts.
        {"name": "experts prompt", "op": "experts", "t": 16384, "e": 16, "n": 4096, "k": 4096, "skew": 0.3, "spare": 0, "type": "bf16"},
        # A training step whose sizes fit no tile and no 16-byte row, with spare rows behind the last group.
        {"name": "experts ragged train", "op": "experts_train", "t": 2047, "e": 11, "n": 1000, "k": 1531, "skew": 1.0, "spare": 33, "type": "f16"},
        # A training step of a large layer.
        {"name": "experts train", "op": "experts_train", "t": 32768, "e": 32, "n": 4096, "k": 2048, "skew": 0.3, "spare": 0, "type": "bf16"},
        # One token while serving: latency alone.
        {"name": "norm token", "op": "norm", "t": 1, "d": 4096, "type": "bf16", "weight": "bf16", "bias": True},
        # A prompt through a wide layer.
        {"name": "norm prompt", "op": "norm", "t": 8192, "d": 8192, "type": "bf16", "weight": "bf16", "bias": False},
        # A training step whose rows have no 16-byte alignment.
        {"name": "norm ragged train", "op": "norm_train", "t": 2047, "d": 1531, "type": "f16", "weight": "f32", "bias": True},
        # A training step with master weights in 32 bits.
        {"name": "norm train", "op": "norm_train", "t": 16384, "d": 4096, "type": "bf16", "weight": "f32", "bias": True},
        # The vectors of a model whose matrices another optimiser updates: many small tensors.
        {"name": "adamw vectors", "op": "adamw", "layers": 24, "d": 1024, "i": 0, "vocab": 0, "param": "f32", "grad": "f32", "copy": None, "bits": 32, "t": 10},
        # All weights of a small model, with the copies that its kernels read.
        {"name": "adamw model", "op": "adamw", "layers": 12, "d": 768, "i": 2048, "vocab": 32003, "param": "f32", "grad": "bf16", "copy": "bf16", "bits": 32, "t": 1000},
        # Weights of large layers, with states in 8 bits.
        {"name": "adamw 8 bit", "op": "adamw", "layers": 2, "d": 4096, "i": 10240, "vocab": 1, "param": "f32", "grad": "bf16", "copy": "bf16", "bits": 8, "t": 1000},
    ]


def _between(rng, lo, hi):
    """A size spread over the logarithm of [lo, hi], odd ones among them."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["experts", "experts", "experts_train", "norm", "norm_train", "adamw", "adamw"])
    while True:
        if op.startswith("experts"):
            # Widths of a layer are multiples of 8 in most models, and anything in the rest.
            step = rng.choice([64, 64, 8, 1])
            case = {"op": op, "t": _between(rng, 1, 32768), "e": _between(rng, 1, 128),
                    "n": max(step, _between(rng, 64, 8192) // step * step),
                    "k": max(step, _between(rng, 64, 8192) // step * step), "skew": rng.choice([0.0, 0.3, 1.0]),
                    "spare": rng.choice([0, 0, _between(rng, 1, 500)]), "type": rng.choice(["bf16", "bf16", "f16"])}
            most = {"bytes": 1.2e9, "flops": 5.6e11} if op == "experts" else {"bytes": 2.4e9, "flops": 1.65e12}
        elif op.startswith("norm"):
            ty = rng.choice(["bf16", "bf16", "f16", "f32"])
            case = {"op": op, "t": _between(rng, 1, 16384), "d": _between(rng, 64, 16384), "type": ty,
                    "weight": rng.choice([ty, "f32"]), "bias": rng.random() < 0.7}
            most = {"bytes": 2.7e8 if op == "norm" else 6.8e8, "flops": 1e99}
        else:
            vectors = rng.random() < 0.25
            param = rng.choice(["f32", "f32", "bf16"])
            case = {"op": op, "layers": rng.randint(1, 24), "d": _between(rng, 64, 4096), "i": 0 if vectors else _between(rng, 128, 10240),
                    "vocab": 0 if vectors else rng.choice([0, _between(rng, 100, 50000)]), "param": param,
                    "grad": rng.choice(["f32", "bf16"]) if param == "f32" else param,
                    "copy": rng.choice([None, "bf16", "f16"]) if param == "f32" else None, "bits": rng.choice([32, 8]),
                    "t": _between(rng, 1, 10000)}
            most = {"bytes": 4.2e9, "flops": 1e99}
        w = work(case)
        # Not above the largest listed case of its operator.
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"]:
            return case


def _sizes(case):
    """Rows of each group: `t` rows sent to experts that are not equally liked."""
    rng = random.Random("%(t)d %(e)d %(skew)r" % case)
    liked = [math.exp(case["skew"] * rng.gauss(0, 1)) for _ in range(case["e"])]
    sizes = [0] * case["e"]
    if case["skew"] == 0 and case["t"] <= case["e"]:
        for e in rng.sample(range(case["e"]), case["t"]):  # one token's experts are different ones
            sizes[e] = 1
    else:
        for e in rng.choices(range(case["e"]), liked, k=case["t"]):
            sizes[e] += 1
    return sizes


def _shapes(case):
    """The tensors of a model: norms of each layer, and its matrices where it has an inner width."""
    d, i, v = case["d"], case["i"], case["vocab"]
    layer = [(d,), (d,)] + ([(2 * i, d), (d, i)] if i else [])
    ends = [(v, d)] if v else []
    return ends + layer * case["layers"] + [(d,), (d,)] + ends


def work(case):
    if case["op"].startswith("experts"):
        e = _SIZE[case["type"]]
        sizes, n, k = _sizes(case), case["n"], case["k"]
        t, rows, used = case["t"], case["t"] + case["spare"], sum(s > 0 for s in sizes)
        forward = e * (t * k + rows * n + used * n * k)
        if case["op"] == "experts":
            return {"bytes": forward, "flops": 2 * t * n * k}
        # Forward and backward share one reading of x and W; dy is read, dx and dW are written.
        return {"bytes": forward + e * (t * n + rows * k + case["e"] * n * k), "flops": 6 * t * n * k}
    if case["op"].startswith("norm"):
        e, w = _SIZE[case["type"]], _SIZE[case["weight"]]
        t, d, vectors = case["t"], case["d"], 2 if case["bias"] else 1
        if case["op"] == "norm":
            return {"bytes": 2 * t * d * e + vectors * d * w, "flops": 8 * t * d}
        # Between the passes lies the rest of the model, so x is read in each.
        return {"bytes": 5 * t * d * e + (2 * vectors + 1) * d * w, "flops": 20 * t * d}
    n = sum(math.prod(s) for s in _shapes(case))
    state = 16 * n if case["bits"] == 32 else 4 * n + 16 * n // _BLOCK
    return {"bytes": n * (2 * _SIZE[case["param"]] + _SIZE[case["grad"]] + _SIZE[case["copy"]]) + state, "flops": 16 * n}


# ----------------------------------------------------------------- inputs --


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale

    s = {"case": dict(case)}
    if case["op"].startswith("experts"):
        dt = _TYPES[case["type"]]
        t, e, n, k = case["t"], case["e"], case["n"], case["k"]
        sizes = _sizes(case)
        random.Random(int(seed)).shuffle(sizes)
        offsets = [0]
        for size in sizes:
            offsets.append(offsets[-1] + size)
        s["offsets"] = torch.tensor(offsets, device="cuda")
        s["most"] = max(sizes)  # the plain form's padding
        s["x"] = normal(t + case["spare"], k).to(dt)
        s["w"] = torch.empty(e, n, k, dtype=dt, device="cuda")
        for i in range(e):
            s["w"][i] = normal(n, k, scale=k ** -0.5)
        if case["op"] == "experts_train":
            s["dy"] = normal(t + case["spare"], n, scale=0.1).to(dt)
    elif case["op"].startswith("norm"):
        dt, wt = _TYPES[case["type"]], _TYPES[case["weight"]]
        t, d = case["t"], case["d"]
        # A residual stream: channels of different size and mean.
        s["x"] = (normal(t, d) * (0.5 + 4.0 * (torch.rand(d, generator=g, device="cuda") > 0.98)) + normal(d, scale=0.3)).to(dt)
        s["weight"] = (1.0 + normal(d, scale=0.1)).to(wt)
        s["bias"] = normal(d, scale=0.1).to(wt) if case["bias"] else None
        if case["op"] == "norm_train":
            s["dy"] = normal(t, d, scale=0.1).to(dt)
    else:
        # Weights, copies and gradients as one buffer each, its tensors at multiples of 256 elements
        # (the states' own layout), and the lists of tensors that a program passes.
        shapes = _shapes(case)
        starts, size = [], 0
        for shape in shapes:
            starts.append(size)
            size += -(-math.prod(shape) // _BLOCK) * _BLOCK
        inside = torch.zeros(size // _BLOCK, _BLOCK, dtype=torch.bool, device="cuda")
        decay = torch.zeros(size // _BLOCK, 1, device="cuda")
        for shape, at in zip(shapes, starts):
            inside.view(-1)[at:at + math.prod(shape)] = True
            decay[at // _BLOCK:-(-(at + math.prod(shape)) // _BLOCK)] = _DECAY if len(shape) > 1 else 0.0

        def views(flat):
            return [flat[at:at + math.prod(shape)].view(shape) for shape, at in zip(shapes, starts)]

        def flat(scale, dtype):
            return (normal(size // _BLOCK, _BLOCK, scale=scale) * inside).view(-1).to(_TYPES[dtype])

        s["decay"], s["decays"] = decay, [_DECAY if len(shape) > 1 else 0.0 for shape in shapes]
        s["param"], s["grad"] = flat(0.02, case["param"]), flat(1e-3, case["grad"])
        s["copy"] = s["param"].to(_TYPES[case["copy"]]) if case["copy"] else None
        s["params"], s["grads"] = views(s["param"]), views(s["grad"])
        s["copies"] = views(s["copy"]) if case["copy"] else None
        s["factor"] = torch.rand((), generator=g, device="cuda") * 0.5 + 0.5  # of a clipped norm
        s["step"] = torch.full((), case["t"] - 1, dtype=torch.int64, device="cuda")
        if case["bits"] == 32:
            s["exp_avg"] = flat(3e-4, "f32")
            s["exp_avg_sq"] = (flat(1e-3, "f32") ** 2 + 1e-7) * inside.view(-1)
            s["scales"] = None
        else:
            blocks = size // _BLOCK
            s["exp_avg"] = (normal(blocks, _BLOCK, scale=120.0).clamp(-448, 448) * inside).view(-1).to(torch.float8_e4m3fn)
            s["exp_avg_sq"] = ((normal(blocks, _BLOCK, scale=120.0).abs() + 1.0).clamp(max=448) * inside).view(-1).to(torch.float8_e4m3fn)
            s["scales"] = torch.exp(normal(2, blocks, scale=0.5)) * torch.tensor([[2.5e-6], [8e-6]], device="cuda")
        if case["t"] == 1:
            for name in ("exp_avg", "exp_avg_sq", "scales"):
                if s[name] is not None:
                    s[name].zero_()
    return s


# ------------------------------------------------------------ plain forms --


def _padded(rows, slots, e, most):
    """Each group's rows as a matrix of `most` rows, filled with zeros."""
    out = torch.zeros(e * most, rows.shape[1], device=rows.device)
    return out.index_copy_(0, slots, rows.float()).view(e, most, -1)


def _plain_experts(s):
    c, dt = s["case"], s["x"].dtype
    t, e, most = c["t"], c["e"], s["most"]
    r = torch.arange(t, device="cuda")
    group = (r.unsqueeze(1) >= s["offsets"][1:]).sum(1)
    slots = group * most + r - s["offsets"][group]
    w = s["w"].float()
    x = _padded(s["x"][:t], slots, e, most)

    def back(padded, width):
        out = torch.zeros(t + c["spare"], width, dtype=dt, device="cuda")
        out[:t] = padded.view(e * most, width)[slots].to(dt)
        return out

    y = back(torch.bmm(x, w.mT), c["n"])
    if c["op"] == "experts":
        return {"y": y}
    dy = _padded(s["dy"][:t], slots, e, most)
    return {"y": y, "dx": back(torch.bmm(dy, w), c["k"]), "dw": torch.bmm(dy.mT, x).to(dt)}


def _plain_norm(s):
    c, dt, wt = s["case"], s["x"].dtype, s["weight"].dtype
    x, w = s["x"].float(), s["weight"].float()
    x = x - x.mean(1, keepdim=True)
    rstd = 1.0 / ((x * x).mean(1, keepdim=True) + _EPS).sqrt()
    xhat = x * rstd
    y = xhat * w
    if c["bias"]:
        y = y + s["bias"].float()
    out = {"y": y.to(dt)}
    if c["op"] == "norm_train":
        dy = s["dy"].float()
        d = dy * w
        out["dx"] = (rstd * (d - d.mean(1, keepdim=True) - xhat * (d * xhat).mean(1, keepdim=True))).to(dt)
        out["dweight"] = (dy * xhat).sum(0).to(wt)
        if c["bias"]:
            out["dbias"] = dy.sum(0).to(wt)
    return out


def _dither(count, t):
    """Evenly spread 20-bit numbers for element j at step t: (a j + b t) mod 1, in 32-bit integers."""
    j = torch.arange(count, dtype=torch.int32, device="cuda")
    a, b = 0xC13FA9A9 - (1 << 32), 0x91E10DA5 - (1 << 32)
    return ((j * a + (t * b).to(torch.int32)) >> 12) & 0xFFFFF


def _plain_adamw(s):
    """All tensors at once, as blocks of 256 of their buffers; the padding between them stays zero."""
    c = s["case"]

    def blocks(v):
        return v.view(-1, _BLOCK)

    s["step"] += 1
    t = s["step"]
    one, two = (1.0 - torch.pow(torch.full((), beta, dtype=torch.float64, device="cuda"), t) for beta in _BETAS)
    p, g = blocks(s["param"]).float(), blocks(s["grad"]).float() * s["factor"]
    m, v = blocks(s["exp_avg"]).float(), blocks(s["exp_avg_sq"]).float()
    if c["bits"] == 8:
        m = m * s["scales"][0].unsqueeze(1)
        v = (v * s["scales"][1].unsqueeze(1)) ** 2
    m = _BETAS[0] * m + (1.0 - _BETAS[0]) * g
    v = _BETAS[1] * v + (1.0 - _BETAS[1]) * (g * g)
    root = v.sqrt()
    p = p - (_LR * s["decay"]) * p - (_LR / one).float() * (m / (root * (1.0 / two.sqrt()).float() + _ADAM_EPS))
    blocks(s["param"]).copy_(p)
    out = {"param": s["param"], "exp_avg": s["exp_avg"], "exp_avg_sq": s["exp_avg_sq"], "step": s["step"]}
    if c["copy"]:
        blocks(s["copy"]).copy_(p)
        out["copy"] = s["copy"]
    if c["bits"] == 32:
        blocks(s["exp_avg"]).copy_(m)
        blocks(s["exp_avg_sq"]).copy_(v)
        return out
    # e4m3 times the block's scale: the average rounded to nearest; of the second moment its root,
    # rounded up or down by the dither, and never from something to nothing.
    scales = torch.stack([m.abs().amax(1), root.amax(1)])
    scales = torch.clamp(scales / 448.0, min=2.0 ** -120)
    m8 = (m * (1.0 / scales[0]).unsqueeze(1)).to(torch.float8_e4m3fn)
    y = torch.clamp(root * (1.0 / scales[1]).unsqueeze(1), max=448.0)
    u = blocks(_dither(y.numel(), t))
    code = torch.where(y < 2.0 ** -6, torch.floor(y * 512.0 + u * 2.0 ** -20).to(torch.int32), ((y.view(torch.int32) + u) >> 20) - 960)
    code = torch.where(root > 0, torch.clamp(code, min=1), code)
    blocks(s["exp_avg"]).copy_(m8)
    blocks(s["exp_avg_sq"]).copy_(code.to(torch.uint8).view(torch.float8_e4m3fn))
    s["scales"].copy_(scales)
    out["scales"] = s["scales"]
    return out


# -------------------------------------------------------------- the calls --


def _own_experts(s):
    import software_pipelined_tiled_gemm_gb300 as sg
    y = sg.grouped_matmul(s["x"], s["w"], s["offsets"])
    if s["case"]["op"] == "experts":
        return {"y": y}
    dx, dw = sg.grouped_matmul_backward(s["dy"], s["x"], s["w"], s["offsets"])
    return {"y": y, "dx": dx, "dw": dw}


def _own_norm(s):
    import software_pipelined_tiled_gemm_gb300 as sg
    if s["case"]["op"] == "norm":
        return {"y": sg.layer_norm(s["x"], s["weight"], s["bias"], eps=_EPS)}
    y, kept = sg.layer_norm(s["x"], s["weight"], s["bias"], eps=_EPS, save=True)
    dx, dweight, dbias = sg.layer_norm_backward(s["dy"], s["x"], s["weight"], kept, need=(True, True, s["case"]["bias"]))
    out = {"y": y, "dx": dx, "dweight": dweight}
    if s["case"]["bias"]:
        out["dbias"] = dbias
    return out


def _own_adamw(s):
    import software_pipelined_tiled_gemm_gb300 as sg
    state = sg.AdamWState(s["step"], s["exp_avg"], s["exp_avg_sq"], s["scales"])
    sg.adamw(s["params"], s["grads"], state, lr=_LR, betas=_BETAS, eps=_ADAM_EPS, weight_decay=s["decays"],
             copies=s["copies"], scale=s["factor"])
    out = {"param": s["param"], "exp_avg": s["exp_avg"], "exp_avg_sq": s["exp_avg_sq"], "step": s["step"]}
    if s["case"]["copy"]:
        out["copy"] = s["copy"]
    if s["case"]["bits"] == 8:
        out["scales"] = s["scales"]
    return out


def run(state):
    op = state["case"]["op"]
    if op.startswith("experts"):
        return _own_experts(state) if own else _plain_experts(state)
    if op.startswith("norm"):
        return _own_norm(state) if own else _plain_norm(state)
    return _own_adamw(state) if own else _plain_adamw(state)


# ----------------------------------------------------- the 64-bit results --


def _to_e4m3(y, u=None):
    """The e4m3 value next to y: the nearest, or with u in [0, 1) the lower one of y + u steps."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    at = y / step
    return ((torch.round(at) if u is None else torch.floor(at + u)) * step).clamp(-448.0, 448.0)


def exact(case, seed):
    """The same outputs in 64 bits; None above a bounded amount of work."""
    if work(case)["flops"] > 5e12:
        return None
    s = prepare(case, seed)
    f = {k: v.double() for k, v in s.items() if torch.is_tensor(v) and v.is_floating_point() and k != "w"}
    if case["op"].startswith("experts"):
        x, w = f["x"], s["w"]
        ends = s["offsets"].tolist()
        y = torch.zeros(x.shape[0], case["n"], dtype=torch.float64, device="cuda")
        out = {"y": y}
        if case["op"] == "experts_train":
            out["dx"] = torch.zeros_like(x)
            out["dw"] = torch.zeros(w.shape, dtype=torch.float64, device="cuda")
        for e in range(case["e"]):
            rows, we = slice(ends[e], ends[e + 1]), w[e].double()
            y[rows] = torch.einsum("rk,nk->rn", x[rows], we)
            if case["op"] == "experts_train":
                out["dx"][rows] = torch.einsum("rn,nk->rk", f["dy"][rows], we)
                out["dw"][e] = torch.einsum("rn,rk->nk", f["dy"][rows], x[rows])
        return out
    if case["op"].startswith("norm"):
        train = case["op"] == "norm_train"
        x, w = f["x"].requires_grad_(train), f["weight"].requires_grad_(train)
        b = f["bias"].requires_grad_(train) if case["bias"] else None
        with torch.enable_grad():
            y = torch.nn.functional.layer_norm(x, (case["d"],), w, b, _EPS)
            if not train:
                return {"y": y}
            grads = torch.autograd.grad(y, [x, w] + ([b] if case["bias"] else []), f["dy"])
        return dict(zip(("dx", "dweight", "dbias"), grads), y=y.detach())
    t = case["t"]
    m, v, g = f["exp_avg"], f["exp_avg_sq"], f["grad"] * f["factor"]
    if case["bits"] == 8:
        m = m * f["scales"][0].repeat_interleave(_BLOCK)
        v = (v * f["scales"][1].repeat_interleave(_BLOCK)).square()
    m = m.lerp(g, 1 - _BETAS[0])
    v = v.lerp(g.square(), 1 - _BETAS[1])
    update = (m / (1 - _BETAS[0] ** t)) / ((v / (1 - _BETAS[1] ** t)).sqrt() + _ADAM_EPS)
    decay = f["decay"].expand(-1, _BLOCK).reshape(-1)
    p = f["param"] * (1 - _LR * decay) - _LR * update
    out = {"param": p, "exp_avg": m, "exp_avg_sq": v, "step": s["step"] + 1}
    if case["copy"]:
        out["copy"] = p
    if case["bits"] == 8:
        root = v.sqrt()
        scales = torch.stack([z.abs().view(-1, _BLOCK).amax(1) for z in (m, root)]).div(448).clamp(min=2.0 ** -120)
        j = torch.arange(p.numel(), device="cuda")
        u = ((j * 0xC13FA9A9 + (t * 0x91E10DA5) % (1 << 32)) % (1 << 32)).div(4096, rounding_mode="floor").double() * 2.0 ** -20
        r8 = _to_e4m3(root / scales[1].repeat_interleave(_BLOCK), u)
        out["exp_avg"] = _to_e4m3(m / scales[0].repeat_interleave(_BLOCK))
        out["exp_avg_sq"] = torch.where(root > 0, r8.clamp(min=2.0 ** -9), r8)
        out["scales"] = scales
    return out


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(n)) for n in range(6)]:
        print(c, work(c))
