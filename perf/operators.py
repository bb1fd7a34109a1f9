"""The cases on which the operators beside the sharded step are measured: AdamW over many tensors,
the embedding with its gradient, and the linear layer in 8-bit floating point.

Where ``own`` is false a case runs in a plain form: elementary torch operations in 32 bits, rounded
once at the end.  Where it is true it makes the calls a user makes of the framework.
"""
import math

import numpy as np
import torch

own = False

BLOCK_STATE = 256   # elements that share a scale in AdamW's 8-bit states
BLOCK_FP8 = 128     # elements that share a scale in the 8-bit matrices
HP = {k: float(np.float32(v)) for k, v in dict(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1).items()}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


# ---- the cases ----------------------------------------------------------------------------------

def listed():
    return [
        # one decoder layer's 11 tensors: a parameter group stepped alone, where launches count
        {"name": "adamw32 one layer", "op": "adamw", "bits": 32, "set": "layers", "n": 1, "d": 512, "ffn": 1024,
         "grad": "f32", "copies": False, "clip": False},
        # tensors of every size, gradients scaled by a clip coefficient on the device
        {"name": "adamw8 ragged", "op": "adamw", "bits": 8, "set": "ragged", "n": 60, "d": 0, "ffn": 0,
         "grad": "f32", "copies": False, "clip": True},
        # a third of the 2048-wide stack: bf16 gradients, fp32 masters, bf16 copies for the forward
        {"name": "adamw32 2048 wide", "op": "adamw", "bits": 32, "set": "layers", "n": 8, "d": 2048, "ffn": 5632,
         "grad": "bf16", "copies": True, "clip": True},
        # half of that stack with 8-bit states, and the states read back as a checkpoint does
        {"name": "adamw8 2048 wide", "op": "adamw", "bits": 8, "set": "layers", "n": 12, "d": 2048, "ffn": 5632,
         "grad": "bf16", "copies": True, "clip": False},
        # the next token of one sequence
        {"name": "lookup one token", "op": "lookup", "tokens": 1, "vocab": 151936, "dim": 1024, "weight": "bf16",
         "out": "bf16", "index": 64},
        # a training batch from fp32 masters, odd vocabulary, rows that no power of two divides
        {"name": "lookup batch", "op": "lookup", "tokens": 16384, "vocab": 32003, "dim": 1000, "weight": "f32",
         "out": "bf16", "index": 32},
        # a small ragged batch's gradient in the parameters' own type
        {"name": "lookup gradient ragged", "op": "lookup_grad", "tokens": 4099, "vocab": 5003, "dim": 517,
         "grad": "bf16", "weight": "bf16", "index": 64, "zipf": False, "accumulate": False},
        # a long batch of text-like token counts into the fp32 main gradient of the 151936-row table
        {"name": "lookup gradient text", "op": "lookup_grad", "tokens": 65536, "vocab": 151936, "dim": 1024,
         "grad": "bf16", "weight": "f32", "index": 64, "zipf": True, "accumulate": False},
        # one token through a projection
        {"name": "linear8 one token", "op": "linear", "m": 1, "n": 2048, "k": 1024, "train": False},
        # a ragged prompt through odd sizes
        {"name": "linear8 ragged prompt", "op": "linear", "m": 333, "n": 1001, "k": 777, "train": False},
        # the 2048-wide stack's feed-forward product in training, weights laid out in the pass
        {"name": "linear8 training", "op": "linear", "m": 8192, "n": 5632, "k": 2048, "train": True},
        # logits of a batch over the whole vocabulary
        {"name": "linear8 logits", "op": "linear", "m": 4096, "n": 151936, "k": 1024, "train": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adamw", "lookup", "lookup_grad", "linear", "linear"])
    if op == "adamw":
        if rng.random() < 0.5:
            d = 64 * rng.randint(4, 32)
            shape = {"set": "layers", "n": rng.randint(1, 12), "d": d, "ffn": d * rng.randint(2, 5) // 2 + rng.randint(0, 9)}
        else:
            shape = {"set": "ragged", "n": rng.randint(1, 100), "d": 0, "ffn": 0}
        return {"op": op, "bits": rng.choice([8, 32]), **shape, "grad": rng.choice(["f32", "bf16"]),
                "copies": rng.random() < 0.5, "clip": rng.random() < 0.5}
    if op == "lookup":
        return {"op": op, "tokens": _log(rng, 1, 32768), "vocab": _log(rng, 1000, 160000), "dim": _log(rng, 64, 3000),
                "weight": rng.choice(["f32", "bf16"]), "out": rng.choice(["f32", "bf16"]), "index": rng.choice([32, 64])}
    if op == "lookup_grad":
        return {"op": op, "tokens": _log(rng, 1, 65536), "vocab": _log(rng, 1000, 150000), "dim": _log(rng, 64, 1024),
                "grad": rng.choice(["f32", "bf16"]), "weight": rng.choice(["f32", "bf16"]), "index": rng.choice([32, 64]),
                "zipf": rng.random() < 0.6, "accumulate": rng.random() < 0.5}
    train = rng.random() < 0.5
    return {"op": op, "m": _log(rng, 1, 8192), "n": _log(rng, 64, 5632 if train else 20000), "k": _log(rng, 64, 4000), "train": train}


def _sizes(case):
    """The elements of each tensor of an AdamW case."""
    d, ffn = case["d"], case["ffn"]
    if case["set"] == "layers":
        return [s for _ in range(case["n"]) for s in (d, d * d, d * d // 4, d * d // 4, d * d, d, ffn * d, ffn * d, d * ffn)]
    r = np.random.RandomState(61557)
    return [int(r.randint(1, 4100)) * int(r.choice([1, 64, 1024, 4096])) for _ in range(case["n"])]


def work(case):
    op = case["op"]
    if op == "adamw":
        n = sum(_sizes(case))
        states = 16 if case["bits"] == 32 else 4 + 16 / BLOCK_STATE + 2 + 8 + 8 / BLOCK_STATE  # 8 bits: and read back as values
        return {"bytes": n * (SIZE[case["grad"]] + 8 + (2 if case["copies"] else 0) + states), "flops": 15 * n}
    if op in ("lookup", "lookup_grad"):
        t, d, v = case["tokens"], case["dim"], case["vocab"]
        if op == "lookup":
            rows = v * (1 - (1 - 1 / v) ** t)   # distinct ones
            return {"bytes": t * case["index"] / 8 + rows * d * SIZE[case["weight"]] + t * d * SIZE[case["out"]], "flops": t * d}
        rows = float(_log_uniform_hit(v, t).sum()) if case["zipf"] else v * (1 - (1 - 1 / v) ** t)
        return {"bytes": t * case["index"] / 8 + t * d * SIZE[case["grad"]] + (2 * rows if case["accumulate"] else v) * d * SIZE[case["weight"]],
                "flops": t * d}
    m, n, k = case["m"], case["n"], case["k"]
    if case["train"]:
        return {"bytes": 2 * (m * k + m * n + n * k) + 2 * m * n + 2 * m * k + 4 * n * k, "flops": 6 * m * n * k}
    return {"bytes": 2 * m * k + n * k * (1 + 1 / BLOCK_FP8) + 2 * m * n, "flops": 2 * m * n * k}


def _log_uniform_hit(v, t):
    """How likely each of v tokens is to be among t log-uniform ones."""
    r = np.arange(1, v + 1)
    return 1 - (1 - np.log1p(1 / r) / math.log(v + 1)) ** t


# ---- what a program has before the call ------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    return {"adamw": _prepare_adamw, "lookup": _prepare_lookup, "lookup_grad": _prepare_lookup_grad,
            "linear": _prepare_linear}[op](case, g)


def _normal(g, shape, std, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _prepare_adamw(case, g):
    sizes = _sizes(case)
    offs, end = [], 0
    for n in sizes:   # each tensor starts a block of its own
        offs.append(end)
        end += -(-n // BLOCK_STATE) * BLOCK_STATE
    inside = torch.zeros(end, device="cuda")
    for o, n in zip(offs, sizes):
        inside[o:o + n] = 1
    s = {"case": case, "t": 9}
    s["p"] = _normal(g, end, 0.02).mul_(inside)
    s["g"] = _normal(g, end, 1e-3).mul_(inside).to(TYPES[case["grad"]])
    s["copy"] = torch.zeros(end, device="cuda", dtype=torch.bfloat16) if case["copies"] else None
    s["clip"] = torch.rand(1, generator=g, device="cuda").mul_(0.5).add_(0.4) if case["clip"] else None
    m = _normal(g, end, 1e-4).mul_(inside)
    v = torch.rand(end, generator=g, device="cuda").square_().mul_(1e-6).mul_(inside)
    if case["bits"] == 32:
        s["m"], s["v"] = m, v
    else:
        s["m"], s["ms"] = _to_codes_m(m)
        s["v"], s["vs"] = _to_codes_v(v)
    if own:
        import fsdp_sharded_mixed_pass_gb300 as fsp
        cut = lambda x: [x[o:o + n] for o, n in zip(offs, sizes)]  # noqa: E731
        opt = fsp.TensorAdamW(cut(s["p"]), cut(s["g"]), copies=None if s["copy"] is None else cut(s["copy"]), lr=HP["lr"],
                              betas=(HP["beta1"], HP["beta2"]), eps=HP["eps"], weight_decay=HP["weight_decay"],
                              state_bits=case["bits"])
        opt.t = s["t"]
        opt.exp_avg.copy_(s["m"])
        opt.exp_avg_sq.copy_(s["v"])
        if case["bits"] == 8:
            opt.exp_avg_scale.copy_(s["ms"])
            opt.exp_avg_sq_scale.copy_(s["vs"])
        s["opt"] = opt
    return s


def _tokens(case, g):
    t, v = case["tokens"], case["vocab"]
    u = torch.rand(t, generator=g, device="cuda", dtype=torch.float64)
    ids = torch.exp(u * math.log(v + 1)) - 1 if case.get("zipf") else u * v
    return ids.floor().clamp_(0, v - 1).to(torch.int32 if case["index"] == 32 else torch.int64)


def _prepare_lookup(case, g):
    return {"case": case, "w": _normal(g, (case["vocab"], case["dim"]), 0.02, TYPES[case["weight"]]), "ids": _tokens(case, g),
            "scale": math.sqrt(case["dim"])}


def _prepare_lookup_grad(case, g):
    s = {"case": case, "ids": _tokens(case, g), "scale": math.sqrt(case["dim"]),
         "dy": _normal(g, (case["tokens"], case["dim"]), 1e-3, TYPES[case["grad"]])}
    shape = (case["vocab"], case["dim"])
    # accumulate: the pass adds to a gradient that an earlier micro-batch left
    s["dw"] = _normal(g, shape, 1e-3, TYPES[case["weight"]]) if case["accumulate"] else torch.empty(shape, device="cuda", dtype=TYPES[case["weight"]])
    return s


def _prepare_linear(case, g):
    m, n, k = case["m"], case["n"], case["k"]
    s = {"case": case, "x": _normal(g, (m, k), 1.0, torch.bfloat16), "w": _normal(g, (n, k), 0.02, torch.bfloat16)}
    if case["train"]:
        s["dy"] = _normal(g, (m, n), 1e-3, torch.bfloat16)
        s["dw"] = torch.empty((n, k), device="cuda")
    if own:
        import fsdp_sharded_mixed_pass_gb300 as fsp
        s["layer"] = fsp.Fp8Linear(s["w"], train=case["train"])
    elif not case["train"]:
        s["codes"] = _quantize(s["w"])   # a serving program lays its weights out once
    return s


# ---- one pass -----------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    return {"adamw": _run_adamw, "lookup": _run_lookup, "lookup_grad": _run_lookup_grad, "linear": _run_linear}[op](state)


def _run_adamw(s):
    case = s["case"]
    if own:
        opt = s["opt"]
        opt.step(grad_scale=s["clip"])
        m, v = opt.state_values() if case["bits"] == 8 else (opt.exp_avg, opt.exp_avg_sq)
    else:
        s["t"] += 1
        m, v = (s["m"], s["v"]) if case["bits"] == 32 else (_from_codes_m(s["m"], s["ms"]), _from_codes_v(s["v"], s["vs"]))
        g = s["g"].float()
        if s["clip"] is not None:
            g = g * s["clip"]
        m = m * HP["beta1"] + g * (1 - HP["beta1"])
        v = v * HP["beta2"] + g * g * (1 - HP["beta2"])
        den = v.sqrt() * (1 / math.sqrt(1 - HP["beta2"] ** s["t"])) + HP["eps"]
        s["p"] = s["p"] * (1 - HP["lr"] * HP["weight_decay"]) - m / den * (HP["lr"] / (1 - HP["beta1"] ** s["t"]))
        if s["copy"] is not None:
            s["copy"] = s["p"].to(torch.bfloat16)
        if case["bits"] == 32:
            s["m"], s["v"] = m, v
        else:
            s["m"], s["ms"] = _to_codes_m(m)
            s["v"], s["vs"] = _to_codes_v(v)
            m, v = _from_codes_m(s["m"], s["ms"]), _from_codes_v(s["v"], s["vs"])
    out = {"p": s["p"], "m": m, "v": v}
    if s["copy"] is not None:
        out["copy"] = s["copy"]
    return out


# the 8-bit states: square-root codes of m and fourth-root codes of v in units of their block's largest

def _to_codes_m(m):
    b = m.view(-1, BLOCK_STATE)
    s = b.abs().amax(1)
    r = (b.abs() / s.where(s > 0, torch.ones_like(s))[:, None]).sqrt() * 127
    return (r.round() * b.sign()).to(torch.int8).view(-1), s


def _from_codes_m(q, s):
    x = q.view(-1, BLOCK_STATE).float() * float(np.float32(1 / 127))
    return (s[:, None] * (x * x.abs())).view(-1)


def _to_codes_v(v):
    b = v.view(-1, BLOCK_STATE)
    s = b.amax(1)
    r = (b / s.where(s > 0, torch.ones_like(s))[:, None]).sqrt().sqrt() * 255
    return torch.maximum(r.round(), (b > 0).float()).to(torch.uint8).view(-1), s


def _from_codes_v(q, s):
    x = q.view(-1, BLOCK_STATE).float() * float(np.float32(1 / 255))
    x = x * x
    return (s[:, None] * (x * x)).view(-1)


def _run_lookup(s):
    if own:
        import fsdp_sharded_mixed_pass_gb300 as fsp
        return fsp.embedding(s["w"], s["ids"], scale=s["scale"], out_dtype=TYPES[s["case"]["out"]])
    return (s["w"][s["ids"]].float() * s["scale"]).to(TYPES[s["case"]["out"]])


def _run_lookup_grad(s):
    case = s["case"]
    if own:
        import fsdp_sharded_mixed_pass_gb300 as fsp
        fsp.embedding_backward(s["ids"], s["dy"], s["dw"], scale=s["scale"], accumulate=case["accumulate"])
        return s["dw"]
    dw = torch.zeros(s["dw"].shape, device="cuda").index_add_(0, s["ids"], s["dy"].float())
    dw = dw * s["scale"]
    s["dw"] = (s["dw"].float() + dw if case["accumulate"] else dw).to(s["dw"].dtype)
    return s["dw"]


def _run_linear(s):
    case = s["case"]
    if own:
        layer = s["layer"]
        if not case["train"]:
            return layer.forward(s["x"])
        layer.update(s["w"])
        y = layer.forward(s["x"])
        dx = layer.backward(s["x"], s["dy"], s["dw"])
        return {"y": y, "dx": dx, "dw": s["dw"]}
    if not case["train"]:
        return (_values(_quantize(s["x"])) @ _values(s["codes"]).t()).to(torch.bfloat16)
    w, wt = _values(_quantize(s["w"])), _values(_quantize(s["w"].t()))
    y = _values(_quantize(s["x"])) @ w.t()
    dx = _values(_quantize(s["dy"])) @ wt.t()
    dw = _values(_quantize(s["dy"].t())) @ _values(_quantize(s["x"].t())).t()
    return {"y": y.to(torch.bfloat16), "dx": dx.to(torch.bfloat16), "dw": dw}


def _blocks(x, dtype):
    """x with its rows cut into blocks, the last one filled up with zeros."""
    r, k = x.shape
    return torch.nn.functional.pad(x.to(dtype), (0, -k % BLOCK_FP8)).view(r, -1, BLOCK_FP8)


def _quantize(x):
    """8-bit codes of x and a power of two for each block of its rows: the smallest with max|x| <= 448 s."""
    b = _blocks(x, torch.float32)
    f, e = torch.frexp(b.abs().amax(2))
    e = (e - 9 + (f > 0.875)).clamp(-127, 127)
    return torch.ldexp(b, -e[:, :, None]).to(torch.float8_e4m3fn), e, x.shape[1]


def _values(q):
    c, e, k = q
    return torch.ldexp(c.float(), e[:, :, None]).flatten(1)[:, :k]


# ---- the definitions in 64 bits ------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"adamw": _exact_adamw, "lookup": _exact_lookup, "lookup_grad": _exact_lookup_grad, "linear": _exact_linear}[case["op"]](case, s)


def _exact_adamw(case, s):
    t = s["t"] + 1
    b1, b2 = HP["beta1"], HP["beta2"]
    g = s["g"].double()
    if s["clip"] is not None:
        g *= s["clip"].double()
    if case["bits"] == 32:
        m, v = s["m"].double(), s["v"].double()
    else:
        up = lambda q, x: x.double().repeat_interleave(BLOCK_STATE) * q  # noqa: E731
        m = up((s["m"].double() / 127).square() * s["m"].sign(), s["ms"])
        v = up((s["v"].double() / 255) ** 4, s["vs"])
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g ** 2
    p = s["p"].double()
    p = p - HP["lr"] * HP["weight_decay"] * p - HP["lr"] * (m / (1 - b1 ** t)) / (torch.sqrt(v / (1 - b2 ** t)) + HP["eps"])
    if case["bits"] == 8:   # what the codes stand for
        def code(x, top, root):
            b = x.abs().unflatten(0, (-1, BLOCK_STATE))
            big = b.amax(1, keepdim=True)
            q = torch.nan_to_num((b / big) ** (1 / root) * top).round()
            if root == 4:
                q = torch.maximum(q, (b > 0).double())
            return ((q / top) ** root * big).flatten() * x.sign()
        m, v = code(m, 127, 2), code(v, 255, 4)
    out = {"p": p, "m": m, "v": v}
    if s["copy"] is not None:
        out["copy"] = p
    return out


def _exact_lookup(case, s):
    return torch.index_select(s["w"], 0, s["ids"]).double() * s["scale"]


def _exact_lookup_grad(case, s):
    order = torch.argsort(s["ids"], stable=True)
    ids, counts = torch.unique_consecutive(s["ids"][order], return_counts=True)
    ends = counts.cumsum(0)
    total = torch.cat([torch.zeros(1, case["dim"], device="cuda", dtype=torch.float64), s["dy"][order].double().cumsum(0)])
    dw = s["dw"].double() if case["accumulate"] else torch.zeros(s["dw"].shape, device="cuda", dtype=torch.float64)
    dw[ids.long()] += (total[ends] - total[ends - counts]) * s["scale"]
    return dw


def _exact_linear(case, s):
    def rounded(x):
        """Each value as its 8-bit code stands for it."""
        b = _blocks(x, torch.float64)
        big = b.abs().amax(2, keepdim=True)
        unit = torch.exp2(torch.ceil(torch.log2(big.clamp_min(2.0 ** -118) / 448)))
        y = b / unit
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
        return ((y / step).round() * step * unit).flatten(1)[:, :x.shape[1]]
    y = rounded(s["x"]) @ rounded(s["w"]).t()
    if not case["train"]:
        return y
    return {"y": y, "dx": rounded(s["dy"]) @ rounded(s["w"].t()).t(), "dw": rounded(s["dy"].t()) @ rounded(s["x"].t()).t()}
