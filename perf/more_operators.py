"""The cases on which the operators between a model's matrix products are measured: layer norm with its
gradients, dropout from a counter-based generator, and rotary positions.

Where ``own`` is false a case runs in a plain form: elementary torch operations in 32 bits (angles and
random words in 64), rounded once at the end.  Where it is true it makes the calls a user makes of the
framework.
"""
import math

import torch

own = False

EPS = 1e-6
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
WORD = 0xFFFFFFFF


# ---- the cases ----------------------------------------------------------------------------------

def listed():
    return [
        # the next token of one sequence, normalised by its root mean square
        {"name": "norm one token", "op": "norm", "rows": 1, "dim": 1024, "x": "bf16", "out": "bf16", "param": "bf16",
         "center": False, "bias": False, "train": False, "add": False},
        # a ragged prompt on an fp32 residual stream, odd rows, with a bias
        {"name": "norm ragged prompt", "op": "norm", "rows": 4099, "dim": 1001, "x": "f32", "out": "bf16", "param": "f32",
         "center": True, "bias": True, "train": False, "add": False},
        # the query heads of 8192 tokens, 16 rows of 128 each: many short rows
        {"name": "norm heads training", "op": "norm", "rows": 131072, "dim": 128, "x": "bf16", "out": "bf16",
         "param": "bf16", "center": False, "bias": False, "train": True, "add": False},
        # the 1024-wide stack's block norm; its gradient joins the residual stream's
        {"name": "norm training 1024 wide", "op": "norm", "rows": 16384, "dim": 1024, "x": "bf16", "out": "bf16",
         "param": "f32", "center": False, "bias": False, "train": True, "add": True},
        # a batch of the 2048-wide stack, centred, with a bias
        {"name": "norm training 2048 wide", "op": "norm", "rows": 32768, "dim": 2048, "x": "bf16", "out": "bf16",
         "param": "f32", "center": True, "bias": True, "train": True, "add": True},
        # a few sequences of the 512-wide layer: a launch's latency
        {"name": "dropout small batch", "op": "dropout", "rows": 64, "dim": 512, "x": "f32", "out": "f32", "p": 0.1,
         "residual": "", "train": False, "device_call": False},
        # odd rows onto an fp32 residual stream, forward pass and gradient; the call's number on the device
        {"name": "dropout ragged training", "op": "dropout", "rows": 3001, "dim": 1001, "x": "bf16", "out": "f32", "p": 0.05,
         "residual": "f32", "train": True, "device_call": True},
        # a batch of the 2048-wide stack onto its residual stream, forward pass and gradient
        {"name": "dropout training", "op": "dropout", "rows": 32768, "dim": 2048, "x": "bf16", "out": "bf16", "p": 0.1,
         "residual": "bf16", "train": True, "device_call": False},
        # the next token of one sequence: 16 query and 8 key heads of 128
        {"name": "rotary one token", "op": "rotary", "batch": 1, "tokens": 1, "heads": 16, "kv": 8, "head_dim": 128,
         "dim": 128, "layout": "half", "x": "bf16", "scaling": "", "factor": 1.0, "start": 4097, "train": False},
        # a ragged prompt, a quarter of each head rotated in pairs, far positions
        {"name": "rotary ragged prompt", "op": "rotary", "batch": 1, "tokens": 1777, "heads": 5, "kv": 1, "head_dim": 80,
         "dim": 20, "layout": "interleaved", "x": "f32", "scaling": "linear", "factor": 8.0, "start": 1000003, "train": False},
        # four sequences of the 1024-wide stack's heads, queries and keys out of one fused projection, both directions
        {"name": "rotary training", "op": "rotary", "batch": 4, "tokens": 4096, "heads": 16, "kv": 8, "head_dim": 128,
         "dim": 128, "layout": "half", "x": "bf16", "scaling": "", "factor": 1.0, "start": 0, "train": True},
        # a long context beyond the trained one, the 512-wide layer's heads
        {"name": "rotary long context", "op": "rotary", "batch": 1, "tokens": 131072, "heads": 8, "kv": 4, "head_dim": 64,
         "dim": 64, "layout": "interleaved", "x": "bf16", "scaling": "yarn", "factor": 4.0, "start": 0, "train": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "dropout", "rotary"])
    largest = max(work(c)["bytes"] for c in listed() if c["op"] == op)
    if op == "norm":
        dim = _log(rng, 32, 16384)
        case = {"op": op, "rows": _log(rng, 1, 131072), "dim": dim if rng.random() < 0.5 else max(32, dim // 32 * 32),
                "x": rng.choice(["f32", "bf16"]), "out": rng.choice(["f32", "bf16"]), "param": rng.choice(["f32", "bf16"]),
                "center": rng.random() < 0.5, "bias": rng.random() < 0.5, "train": rng.random() < 0.6,
                "add": rng.random() < 0.5}
    elif op == "dropout":
        dim = _log(rng, 32, 16384)
        case = {"op": op, "rows": _log(rng, 1, 65536), "dim": dim if rng.random() < 0.5 else max(32, dim // 32 * 32),
                "x": rng.choice(["f32", "bf16"]), "out": rng.choice(["f32", "bf16"]), "p": rng.choice([0.02, 0.05, 0.1, 0.2, 0.5]),
                "residual": rng.choice(["", "f32", "bf16"]), "train": rng.random() < 0.6, "device_call": rng.random() < 0.5}
    else:
        head_dim = rng.choice([32, 48, 64, 80, 96, 128, 192, 256, 2 * rng.randint(8, 128)])
        case = {"op": op, "batch": rng.randint(1, 4), "tokens": _log(rng, 1, 131072), "heads": rng.randint(1, 32),
                "kv": rng.randint(1, 8), "head_dim": head_dim,
                "dim": head_dim if rng.random() < 0.5 else 2 * rng.randint(4, head_dim // 2),
                "layout": rng.choice(["half", "interleaved"]), "x": rng.choice(["f32", "bf16"]),
                "scaling": rng.choice(["", "linear", "ntk", "yarn"]), "factor": float(rng.choice([2, 4, 8, 32])),
                "start": rng.choice([0, 0, _log(rng, 1, 4000000)]), "train": rng.random() < 0.5}
    long = "tokens" if op == "rotary" else "rows"
    while work(case)["bytes"] > largest:
        case[long] = max(1, case[long] * 2 // 3)
    return case


def work(case):
    op = case["op"]
    if op == "rotary":
        rows = case["batch"] * case["tokens"]
        n = rows * (case["heads"] + case["kv"])
        passes = 2 if case["train"] else 1
        return {"bytes": passes * (2 * n * case["head_dim"] * SIZE[case["x"]] + 8 * case["tokens"]),
                "flops": passes * (3 * n * case["dim"] + 2 * rows * case["dim"])}
    n, sx, so = case["rows"] * case["dim"], SIZE[case["x"]], SIZE[case["out"]]
    if op == "dropout":
        moved = n * (sx + so + SIZE.get(case["residual"], 0)) + (n * (so + sx) if case["train"] else 0)
        return {"bytes": moved, "flops": (2 if case["train"] else 1) * 2 * n}
    params = (2 if case["bias"] else 1) * case["dim"]
    bytes_, flops = n * (sx + so) + params * SIZE[case["param"]], 7 * n
    if case["train"]:
        bytes_ += n * (sx + so + sx + (sx if case["add"] else 0)) + 16 * case["rows"] + case["dim"] * SIZE[case["param"]] + 8 * params
        flops += 14 * n
    return {"bytes": bytes_, "flops": flops}


# ---- what a program has before the call ------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"norm": _prepare_norm, "dropout": _prepare_dropout, "rotary": _prepare_rotary}[case["op"]](case, g)


def _normal(g, shape, std, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _prepare_norm(case, g):
    rows, dim, param = case["rows"], case["dim"], TYPES[case["param"]]
    # a residual stream: columns of unlike spread around means of their own
    x = _normal(g, (rows, dim), 1.0).mul_(torch.exp(_normal(g, dim, 0.5))).add_(_normal(g, dim, 0.3))
    s = {"case": case, "x": x.to(TYPES[case["x"]]), "w": _normal(g, dim, 0.2).add_(1).to(param),
         "b": _normal(g, dim, 0.1, param) if case["bias"] else None}
    if case["train"]:
        s["dy"] = _normal(g, (rows, dim), 1e-3, TYPES[case["out"]])
        s["add"] = _normal(g, (rows, dim), 1e-3, TYPES[case["x"]]) if case["add"] else None
        # main gradients that an earlier micro-batch left
        s["dw"] = _normal(g, dim, 1e-3)
        s["db"] = _normal(g, dim, 1e-3) if case["bias"] else None
    return s


def _prepare_dropout(case, g):
    rows, dim = case["rows"], case["dim"]
    seed, call = (int(v) for v in torch.randint(0, 2 ** 62, (2,), generator=g, device="cuda").cpu())
    s = {"case": case, "x": _normal(g, (rows, dim), 1.0, TYPES[case["x"]]), "seed": seed, "call": call,
         "h": _normal(g, (rows, dim), 3.0, TYPES[case["residual"]]) if case["residual"] else None}
    if case["device_call"]:
        s["call"] = torch.full((1,), call, device="cuda", dtype=torch.int64)
    if case["train"]:
        s["dy"] = _normal(g, (rows, dim), 1e-3, TYPES[case["out"]])
    return s


def _prepare_rotary(case, g):
    b, t, h, kv, d = case["batch"], case["tokens"], case["heads"], case["kv"], case["head_dim"]
    qkv = _normal(g, (b, t, h + 2 * kv, d), 1.0, TYPES[case["x"]])
    s = {"case": case, "q": qkv[:, :, :h], "k": qkv[:, :, h:h + kv], "pos": torch.arange(t, device="cuda") + case["start"]}
    if case["train"]:
        s["dq"] = _normal(g, (b, t, h, d), 1e-3, TYPES[case["x"]])
        s["dk"] = _normal(g, (b, t, kv, d), 1e-3, TYPES[case["x"]])
    if own:
        import fsdp_sharded_mixed_pass_gb300 as fsp
        s["rope"] = fsp.Rotary(case["dim"], base=10000.0, layout=case["layout"], scaling=case["scaling"] or None,
                               factor=case["factor"], original_length=4096)
    else:
        s["freq"], s["scale"] = _frequencies(case)   # a program keeps them
    return s


# ---- one pass -----------------------------------------------------------------------------------------

def run(state):
    return {"norm": _run_norm, "dropout": _run_dropout, "rotary": _run_rotary}[state["case"]["op"]](state)


def _run_norm(s):
    case = s["case"]
    out = TYPES[case["out"]]
    if own:
        import fsdp_sharded_mixed_pass_gb300 as fsp
        if not case["train"]:
            return fsp.layer_norm(s["x"], s["w"], s["b"], eps=EPS, center=case["center"], out_dtype=out)
        y, stats = fsp.layer_norm(s["x"], s["w"], s["b"], eps=EPS, center=case["center"], out_dtype=out, stats=True)
        dx = fsp.layer_norm_backward(s["x"], stats, s["dy"], s["w"], center=case["center"], grad_weight=s["dw"],
                                     grad_bias=s["db"], accumulate=True, add=s["add"])
    else:
        x, w = s["x"].float(), s["w"].float()
        if case["center"]:
            x = x - x.mean(1, keepdim=True)
        r = 1 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
        xhat = x * r
        y = xhat * w
        if case["bias"]:
            y = y + s["b"].float()
        y = y.to(out)
        if not case["train"]:
            return y
        dy = s["dy"].float()
        s["dw"] = s["dw"] + (dy * xhat).sum(0)
        if case["bias"]:
            s["db"] = s["db"] + dy.sum(0)
        g = dy * w
        dx = g - xhat * (g * xhat).mean(1, keepdim=True)
        if case["center"]:
            dx = dx - g.mean(1, keepdim=True)
        dx = dx * r
        if case["add"]:
            dx = dx + s["add"].float()
        dx = dx.to(s["x"].dtype)
    got = {"y": y, "dx": dx, "dw": s["dw"]}
    if case["bias"]:
        got["db"] = s["db"]
    return got


def _run_dropout(s):
    case = s["case"]
    out, p = TYPES[case["out"]], case["p"]
    if own:
        import fsdp_sharded_mixed_pass_gb300 as fsp
        y = fsp.dropout(s["x"], p, s["seed"], s["call"], residual=s["h"], out_dtype=out)
        if not case["train"]:
            return y
        return {"y": y, "dx": fsp.dropout_backward(s["dy"], p, s["seed"], s["call"], out_dtype=s["x"].dtype)}
    shape = s["x"].shape
    dropped = int(p * 65536 + 0.5)   # of 65536: an element goes where its 16 random bits are below
    keep = (_random16(s["x"].numel(), s["seed"], s["call"]) >= dropped).view(shape)
    scale = 65536 / (65536 - dropped)
    y = torch.where(keep, s["x"].float() * scale, 0.0)
    if s["h"] is not None:
        y = y + s["h"].float()
    y = y.to(out)
    if not case["train"]:
        return y
    keep = (_random16(s["x"].numel(), s["seed"], s["call"]) >= dropped).view(shape)   # no mask is kept
    return {"y": y, "dx": torch.where(keep, s["dy"].float() * scale, 0.0).to(s["x"].dtype)}


def _random16(n, seed, call):
    """n random numbers of 16 bits: Philox-4x32 of ten rounds (Salmon, Moraes, Dror and Shaw, "Parallel random
    numbers: as easy as 1, 2, 3", 2011), keyed by the seed; its counter is the number's index / 8 and the call,
    and its four words give eight numbers, each word's lower half first."""
    i = torch.arange((n + 7) // 8, device="cuda")
    call = torch.as_tensor(call, device="cuda", dtype=torch.int64)
    a, b, c, d = i & WORD, i >> 32, (call & WORD).expand(i.shape), (call >> 32 & WORD).expand(i.shape)
    k0, k1 = seed & WORD, seed >> 32 & WORD
    for r in range(10):
        u, v = a * 0xD2511F53, c * 0xCD9E8D57   # (64 bits; the sign is cut off with the shift)
        a, b, c, d = (v >> 32 & WORD) ^ b ^ (k0 + r * 0x9E3779B9 & WORD), v & WORD, (u >> 32 & WORD) ^ d ^ (k1 + r * 0xBB67AE85 & WORD), u & WORD
    words = torch.stack([a, b, c, d], 1)
    return torch.stack([words & 0xFFFF, words >> 16], 2).view(-1)[:n]


def _frequencies(case):
    """Radians per position of each pair, and what the rotated elements are multiplied by."""
    d, base, factor = case["dim"], 10000.0, case["factor"]
    if case["scaling"] == "ntk" and d > 2:
        base = base * factor ** (d / (d - 2))
    f = base ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)
    if case["scaling"] == "linear":
        return f / factor, 1.0
    if case["scaling"] != "yarn":
        return f, 1.0
    # pairs that turn more than 32 times over the trained length stay, those below one turn are stretched (Peng, Quesnelle,
    # Fan and Shippole, "YaRN: Efficient context window extension of large language models", 2023)
    kept = ((f * 4096 / (2 * math.pi) - 1) / 31).clamp(0, 1)
    return f / factor * (1 - kept) + f * kept, 0.1 * math.log(factor) + 1


def _run_rotary(s):
    case = s["case"]
    if own:
        rope = s["rope"]
        q, k = rope.forward((s["q"], s["k"]), s["pos"])
        if not case["train"]:
            return {"q": q, "k": k}
        dq, dk = rope.backward((s["dq"], s["dk"]), s["pos"])
        return {"q": q, "k": k, "dq": dq, "dk": dk}
    angle = s["pos"].double()[:, None] * s["freq"]
    c, w = (torch.cos(angle) * s["scale"]).float(), (torch.sin(angle) * s["scale"]).float()
    got = {"q": _rotate(case, s["q"], c, w), "k": _rotate(case, s["k"], c, w)}
    if case["train"]:
        got["dq"], got["dk"] = _rotate(case, s["dq"], c, -w), _rotate(case, s["dk"], c, -w)
    return got


def _rotate(case, x, c, w):
    """The first elements of each head as pairs turned by angles of cosine c and sine w (tokens x pairs)."""
    dim, dtype = case["dim"], x.dtype
    c, w = c[:, None], w[:, None]   # for every head
    out = x.float().clone()
    first, second = (slice(0, dim // 2), slice(dim // 2, dim)) if case["layout"] == "half" else (slice(0, dim, 2), slice(1, dim, 2))
    a, b = x[..., first].float(), x[..., second].float()
    out[..., first] = a * c - b * w
    out[..., second] = b * c + a * w
    return out.to(dtype)


# ---- the definitions in 64 bits ------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "dropout": _exact_dropout, "rotary": _exact_rotary}[case["op"]](case, s)


def _exact_norm(case, s):
    """The forward pass by its definition; the gradients by differentiating it."""
    x, w = s["x"].double().requires_grad_(case["train"]), s["w"].double().requires_grad_(case["train"])
    b = s["b"].double().requires_grad_(case["train"]) if case["bias"] else None
    if case["center"]:
        var, mean = torch.var_mean(x, 1, unbiased=False, keepdim=True)
        y = (x - mean) * torch.rsqrt(var + EPS) * w
    else:
        y = x * torch.rsqrt(x.pow(2).mean(1, keepdim=True) + EPS) * w
    if b is not None:
        y = y + b
    if not case["train"]:
        return y
    y.backward(s["dy"].double())
    got = {"y": y.detach(), "dx": x.grad + s["add"] if case["add"] else x.grad, "dw": s["dw"] + w.grad}
    if b is not None:
        got["db"] = s["db"] + b.grad
    return got


def _exact_dropout(case, s):
    n = s["x"].numel()
    lost = int(round(case["p"] * 65536))
    keep = (_halfwords(n, s["seed"], int(s["call"])) >= lost).view(s["x"].shape)
    y = s["x"].double() * keep * (65536 / (65536 - lost))
    if s["h"] is not None:
        y += s["h"]
    return {"y": y, "dx": s["dy"].double() * keep * (65536 / (65536 - lost))} if case["train"] else y


def _halfwords(n, seed, call):
    """The generator's numbers, its words held as halves of 16 bits: [count, 2], the lower half first."""
    count = (n + 7) // 8
    halves = lambda v: torch.stack([v & 0xFFFF, v >> 16 & 0xFFFF], -1)  # noqa: E731
    i = torch.arange(count, device="cuda")
    constant = lambda v: halves(torch.tensor(v, device="cuda")).expand(count, 2)  # noqa: E731
    x = [halves(i), halves(i >> 32), constant(call & WORD), constant(call >> 32 & WORD)]
    key = [seed & WORD, seed >> 32 & WORD]

    def product(v, m):   # (upper word, lower word) of a word times a constant, by schoolbook
        p0 = v[:, 0] * (m & 0xFFFF)
        p1 = v[:, 1] * (m & 0xFFFF) + (p0 >> 16)
        q0 = v[:, 0] * (m >> 16) + (p1 & 0xFFFF)
        q1 = v[:, 1] * (m >> 16) + (p1 >> 16) + (q0 >> 16)
        return halves(q1), torch.stack([p0 & 0xFFFF, q0 & 0xFFFF], -1)

    for _ in range(10):
        hi0, lo0 = product(x[0], 0xD2511F53)
        hi1, lo1 = product(x[2], 0xCD9E8D57)
        x = [hi1 ^ x[1] ^ constant(key[0]), lo1, hi0 ^ x[3] ^ constant(key[1]), lo0]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    return torch.cat(x, 1).flatten()[:n]


def _exact_rotary(case, s):
    """Pairs as complex numbers, times a complex number of the position's angle."""
    d, n = case["dim"], case["dim"] // 2
    freq = []
    for j in range(n):
        base = 10000.0 * case["factor"] ** (d / (d - 2)) if case["scaling"] == "ntk" and d > 2 else 10000.0
        f = math.exp(-2 * j / d * math.log(base))
        if case["scaling"] == "linear":
            f /= case["factor"]
        if case["scaling"] == "yarn":
            turns = 4096 * f / math.tau
            part = 1.0 if turns > 32 else 0.0 if turns < 1 else (turns - 1) / 31
            f = part * f + (1 - part) * f / case["factor"]
        freq.append(f)
    scale = 1 + 0.1 * math.log(case["factor"]) if case["scaling"] == "yarn" else 1.0
    turn = torch.polar(torch.full((case["tokens"], n), scale, device="cuda", dtype=torch.float64),
                       torch.outer(s["pos"].double(), torch.tensor(freq, device="cuda", dtype=torch.float64)))[:, None]

    def turned(x, by):
        x = x.double()
        head, rest = x[..., :d], x[..., d:]
        pairs = head.unflatten(-1, (2, n)).transpose(-1, -2) if case["layout"] == "half" else head.unflatten(-1, (n, 2))
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * by)
        z = z.transpose(-1, -2).flatten(-2) if case["layout"] == "half" else z.flatten(-2)
        return torch.cat([z, rest], -1)

    got = {"q": turned(s["q"], turn), "k": turned(s["k"], turn)}
    if case["train"]:
        got["dq"], got["dk"] = turned(s["dq"], turn.conj()), turned(s["dk"], turn.conj())
    return got
