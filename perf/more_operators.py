"""The cases that the linear, AdamW and mixture-of-experts operators are measured on.

`linear_forward` and `linear_backward` (a product with bias, activation and
residual in its epilogue, and its gradients), `AdamW` (a step over many tensors
at once with moments in 32 or 8 bits) and `moe` (a mixture-of-experts layer for a few tokens: router,
choice, gated experts, weighted sum).  `run` computes either their plain form (elementary
torch operations, rounded once) or calls the package, by `own`.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BLOCK = 256     # entries that share one exponent in 8-bit moments
LR, BETAS, EPS, DECAY = 1e-3, (0.9, 0.95), 1e-8, 0.1


def listed():
    return [
        # the down projection of a 4B-class layer, one token, added to the residual stream: latency counts
        {"name": "linear_2560x9728_t1", "op": "linear", "rows": 2560, "cols": 9728, "tokens": 1, "dtype": "bf16",
         "act": "none", "bias": False, "residual": True},
        # a biased projection with its activation, a small batch on odd sizes
        {"name": "linear_3001x1237_t7", "op": "linear", "rows": 3001, "cols": 1237, "tokens": 7, "dtype": "f16",
         "act": "gelu", "bias": True, "residual": False},
        # the down projection of a prompt or a calibration batch
        {"name": "linear_2560x9728_t4096", "op": "linear", "rows": 2560, "cols": 9728, "tokens": 4096, "dtype": "bf16",
         "act": "none", "bias": False, "residual": True},
        # a training step's share of the down projection: forward, then every gradient
        {"name": "lintrain_2560x9728_t2048", "op": "lintrain", "rows": 2560, "cols": 9728, "tokens": 2048,
         "dtype": "bf16", "act": "none", "bias": False, "residual": True},
        # a training step of an ungated layer on a ragged batch and odd sizes
        {"name": "lintrain_1001x1237_t777", "op": "lintrain", "rows": 1001, "cols": 1237, "tokens": 777,
         "dtype": "f16", "act": "gelu_tanh", "bias": True, "residual": True},
        # norms and biases, or a few small adapters: latency counts
        {"name": "adamw_small_32", "op": "adamw", "matrices": 2, "rows": 16, "cols": 2560, "vectors": 4, "bits": 32,
         "dtype": "bf16", "grad": "bf16", "master": True},
        # the three matrices of a 4B-class feed-forward block with fp32 master weights
        {"name": "adamw_block_32", "op": "adamw", "matrices": 3, "rows": 9728, "cols": 2560, "vectors": 2, "bits": 32,
         "dtype": "bf16", "grad": "bf16", "master": True},
        # the same with moments in 8 bits
        {"name": "adamw_block_8", "op": "adamw", "matrices": 3, "rows": 9728, "cols": 2560, "vectors": 2, "bits": 8,
         "dtype": "bf16", "grad": "bf16", "master": True},
        # many tensors of odd sizes in one flat buffer, without master weights
        {"name": "adamw_ragged_8", "op": "adamw", "matrices": 9, "rows": 1001, "cols": 1237, "vectors": 5, "bits": 8,
         "dtype": "f16", "grad": "f32", "master": False},
        # one token through a mixture of 64 experts
        {"name": "moe_e64_k4_t1", "op": "moe", "experts": 64, "top": 4, "rows": 1024, "cols": 2560, "tokens": 1,
         "dtype": "bf16", "act": "silu", "normalize": True},
        # a small batch on odd sizes, weights of the softmax over all experts
        {"name": "moe_e13_k3_t7", "op": "moe", "experts": 13, "top": 3, "rows": 701, "cols": 1237, "tokens": 7,
         "dtype": "f16", "act": "gelu", "normalize": False},
        # 32 sequences, one token each: most of the 128 experts are read
        {"name": "moe_e128_k8_t32", "op": "moe", "experts": 128, "top": 8, "rows": 768, "cols": 2560, "tokens": 32,
         "dtype": "bf16", "act": "silu", "normalize": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A matrix dimension: mostly a multiple of 64, as models have them, else any."""
    n = _log_int(rng, lo, hi)
    return max(64, (n + 32) // 64 * 64) if rng.random() < 0.6 else n


def draw(rng):
    op = rng.choice(["linear", "lintrain", "adamw", "adamw", "moe", "moe"])
    case = {"op": op}
    if op == "adamw":
        case["rows"], case["cols"] = _size(rng, 16, 9728), _size(rng, 64, 9728)
        case["matrices"] = rng.randint(1, 12)
        while case["matrices"] > 1 and case["matrices"] * case["rows"] * case["cols"] > 3 * 9728 * 2560:
            case["matrices"] -= 1
        case["rows"] = min(case["rows"], 3 * 9728 * 2560 // case["cols"])
        case["vectors"] = rng.randint(0, 6)
        case["bits"] = rng.choice([8, 32])
        case["dtype"], case["grad"] = rng.choice(["bf16", "f16", "f32"]), rng.choice(["bf16", "f16", "f32"])
        case["master"] = case["dtype"] != "f32" and rng.random() < 0.7
        return case
    case["dtype"] = rng.choice(["bf16", "f16"])
    if op == "moe":
        case["experts"] = _log_int(rng, 4, 128)
        case["top"] = rng.randint(1, min(8, case["experts"]))
        case["rows"], case["cols"] = _size(rng, 64, 2048), _size(rng, 256, 4096)
        case["tokens"] = _log_int(rng, 1, 64)
        while case["experts"] * case["rows"] * case["cols"] > 128 * 768 * 2560:
            case["rows"] //= 2
        most = 32 * 8 * 768 * 2560
        case["tokens"] = max(1, min(case["tokens"], most // (case["top"] * case["rows"] * case["cols"])))
        case["act"] = rng.choice(["silu", "gelu", "gelu_tanh"])
        case["normalize"] = rng.random() < 0.7
        return case
    case["rows"], case["cols"] = _size(rng, 256, 9728), _size(rng, 256, 9728)
    case["tokens"] = _log_int(rng, 1, 4096)
    most = 9728 * 2560 * (2048 if op == "lintrain" else 4096) // (1 if op == "linear" else 2)
    case["tokens"] = max(1, min(case["tokens"], most // (case["rows"] * case["cols"])))
    case["act"] = rng.choice(["none", "silu", "gelu", "gelu_tanh"])
    case["bias"], case["residual"] = rng.random() < 0.5, rng.random() < 0.5
    return case


# ---------------------------------------------------------------- inputs

def _activations(tokens, cols, normal, gen, dtype):
    """Normalised activations with a few strong channels."""
    x = normal(tokens, cols)
    x[:, torch.randperm(cols, generator=gen, device="cuda")[:4]] *= 4.0
    return x.to(dtype)


def _sizes(case):
    return [case["rows"] * case["cols"]] * case["matrices"] + [case["cols"]] * case["vectors"]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")
    dtype = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "adamw":
        _prepare_adamw(s, normal, dtype)
        return s
    rows, cols, tokens = case["rows"], case["cols"], case["tokens"]
    s["x"] = _activations(tokens, cols, normal, gen, dtype)
    if case["op"] == "moe":
        experts = case["experts"]
        s["wr"] = (normal(experts, cols) / math.sqrt(cols)).to(dtype)
        # gate and up rows of an expert lie one after the other, as checkpoints keep them
        both = torch.empty(experts, 2 * rows, cols, dtype=dtype, device="cuda")
        s["wd"] = torch.empty(experts, cols, rows, dtype=dtype, device="cuda")
        for e in range(experts):
            both[e] = normal(2 * rows, cols) / math.sqrt(cols)
            s["wd"][e] = normal(cols, rows) / math.sqrt(rows)
        s["wg"], s["wu"] = both[:, :rows], both[:, rows:]
        return s
    s["w"] = (normal(rows, cols) / math.sqrt(cols)).to(dtype)
    s["bias"] = (0.5 * normal(rows)).to(dtype) if case["bias"] else None
    s["residual"] = normal(tokens, rows).to(dtype) if case["residual"] else None
    if case["op"] == "lintrain":
        s["dy"] = normal(tokens, rows).to(dtype)
    return s


def _prepare_adamw(s, normal, dtype):
    """Parameters, gradients and state of a run's 100th step.  Parameters and gradients are pieces of one flat
    buffer; the state has each tensor's entries filled up with zeros to whole blocks, one tensor after the other."""
    case = s["case"]
    sizes = s["sizes"] = _sizes(case)
    total = sum(sizes)
    weights = 0.02 * normal(total)
    master = weights.to(dtype).float() + 1e-5 * normal(total)
    s["flat"] = (master if case["master"] else weights).to(dtype)
    s["grad"] = (1e-3 * normal(total)).to(DTYPES[case["grad"]])
    s["params"], s["grads"] = list(s["flat"].split(sizes)), list(s["grad"].split(sizes))
    # moments of gradients that differ in size from one part of a tensor to another
    size = 1e-3 * torch.exp(2.0 * normal(-(-total // 64))).repeat_interleave(64)[:total]
    m, v = 0.3 * size * normal(total), size * size * (0.1 + normal(total).square())
    m, v = _filled(m, sizes), _filled(v, sizes)
    step = torch.tensor([99.0, BETAS[0] ** 99, BETAS[1] ** 99, 0.0], dtype=torch.float64, device="cuda")
    s["state"] = {"step": step, "m": m if case["bits"] == 32 else _encode_m(m),
                  "v": v if case["bits"] == 32 else _encode_v(v), "master": _filled(master, sizes) if case["master"] else None}


def _filled(flat, sizes):
    """A flat buffer's pieces, each filled up to whole blocks."""
    return torch.cat([torch.nn.functional.pad(t, (0, -t.numel() % BLOCK)) for t in flat.split(sizes)])


def _unfilled(padded, sizes):
    pieces = padded.split([-(-n // BLOCK) * BLOCK for n in sizes])
    return torch.cat([t[:n] for t, n in zip(pieces, sizes)])


# 8-bit moments: a byte per entry, then a byte per block, the exponent field of the block's largest
# magnitude (15 at least).

def _exponents(blocks):
    return (blocks.abs().amax(1, keepdim=True).view(torch.int32) >> 23).clamp(min=15)


def _encode_m(t):
    """An OCP e4m3 number times 2^(b - 134), b the block's byte."""
    t = t.view(-1, BLOCK)
    b = _exponents(t)
    code = (t * ((261 - b) << 23).view(torch.float32)).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.cat([code.view(-1), b.to(torch.uint8).view(-1)])


def _parts(buffer):
    blocks = buffer.numel() // (BLOCK + 1)
    return buffer[:blocks * BLOCK].view(-1, BLOCK), buffer[blocks * BLOCK:].view(-1, 1).int()


def _decode_m(buffer):
    code, b = _parts(buffer)
    return (code.view(torch.float8_e4m3fn).float() * ((b - 7) << 23).view(torch.float32)).view(-1)


def _encode_v(t):
    """Five bits of exponent and three of mantissa, no sign, times 2^(b - 141); what is not 0 does not become 0."""
    t = t.view(-1, BLOCK)
    b = _exponents(t)
    t = t * ((268 - b) << 23).view(torch.float32)
    bits = t.view(torch.int32)
    normal = ((bits + 0x7ffff + ((bits >> 20) & 1)) >> 20) - (112 << 3)
    code = torch.where(t < 2.0 ** -14, torch.round(t * 2.0 ** 17).int().clamp(min=1), normal)
    return torch.cat([torch.where(t > 0, code, 0).to(torch.uint8).view(-1), b.to(torch.uint8).view(-1)])


def _decode_v(buffer):
    code, b = _parts(buffer)
    code = code.int()
    value = torch.where(code < 8, code.float() * 2.0 ** -17, ((code + (112 << 3)) << 20).view(torch.float32))
    return (value * ((b - 14) << 23).view(torch.float32)).view(-1)


# ---------------------------------------------------------------- one pass

def _act(g, act):
    if act == "none":
        return g
    if act == "silu":
        return g / (1 + torch.exp(-g))
    if act == "gelu":
        return 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5)))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))


def _act_slope(g, act):
    if act == "silu":
        p = 1 / (1 + torch.exp(-g))
        return p * (1 + g * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    t = torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g))
    return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g * g)


def _plain_linear(s):
    case, dtype = s["case"], s["x"].dtype
    x, w = s["x"].float(), s["w"].float()
    z = x @ w.t()
    if case["bias"]:
        z = z + s["bias"].float()
    y = _act(z, case["act"])
    if case["residual"]:
        y = y + s["residual"].float()
    y = y.to(dtype)
    if case["op"] == "linear":
        return y
    dz = s["dy"].float()
    if case["act"] != "none":
        dz = dz * _act_slope(z, case["act"])
    return {"y": y, "dx": (dz @ w).to(dtype), "dw": (dz.t() @ x).to(dtype),
            "db": dz.sum(0).to(dtype) if case["bias"] else None}


def _plain_adamw(s):
    case, state, sizes = s["case"], s["state"], s["sizes"]
    step, eight = state["step"], case["bits"] == 8
    step[0] += 1
    step[1] *= BETAS[0]
    step[2] *= BETAS[1]
    rate = (LR / (1 - step[1])).float()
    root = (1 - step[2]).rsqrt().float()
    g = _filled(s["grad"].float(), sizes)
    m, v = (_decode_m(state["m"]), _decode_v(state["v"])) if eight else (state["m"], state["v"])
    m = BETAS[0] * m + (1 - BETAS[0]) * g
    v = BETAS[1] * v + (1 - BETAS[1]) * (g * g)
    p = state["master"] if case["master"] else _filled(s["flat"].float(), sizes)
    p = (1 - LR * DECAY) * p - rate * (m / (v.sqrt() * root + EPS))
    s["flat"].copy_(_unfilled(p, sizes))
    if case["master"]:
        state["master"].copy_(p)
    state["m"].copy_(_encode_m(m) if eight else m)
    state["v"].copy_(_encode_v(v) if eight else v)
    return _adamw_outputs(s, (_decode_m(state["m"]), _decode_v(state["v"])) if eight else (state["m"], state["v"]))


def _adamw_outputs(s, moments):
    return {"params": s["flat"], "master": s["state"]["master"], "m": moments[0], "v": moments[1]}


def _plain_moe(s):
    case, dtype, x = s["case"], s["x"].dtype, s["x"].float()
    top, cols = case["top"], case["cols"]
    # the choice is a comparison: in 64 bits
    logits = s["x"].double() @ s["wr"].double().t()
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    ids, chosen = order.indices[:, :top], order.values[:, :top]
    e = torch.exp(chosen - order.values[:, :1])
    weights = (e / (e if case["normalize"] else torch.exp(logits - order.values[:, :1])).sum(1, keepdim=True)).float()
    # every chosen expert's matrices, one copy per slot
    slots = ids.reshape(-1)
    xs = x.repeat_interleave(top, 0).view(-1, cols, 1)
    g, u = torch.matmul(s["wg"][slots].float(), xs), torch.matmul(s["wu"][slots].float(), xs)
    y = torch.matmul(s["wd"][slots].float(), _act(g, case["act"]) * u)
    y = (y.view(-1, top, cols) * weights[..., None]).sum(1).to(dtype)
    return {"y": y, "ids": ids.int(), "weights": weights}


def _own(s):
    import ternary_rank_weight_amd as trw
    case = s["case"]
    op = case["op"]
    if op == "moe":
        y, ids, weights = trw.moe(s["x"], s["wr"], s["wg"], s["wu"], s["wd"], case["top"], case["act"],
                                  normalize=case["normalize"], routing=True)
        return {"y": y, "ids": ids, "weights": weights}
    if op == "adamw":
        if "opt" not in s:   # the optimizer that a program keeps
            s["opt"] = trw.AdamW(s["params"], lr=LR, betas=BETAS, eps=EPS, weight_decay=DECAY, bits=case["bits"],
                                 master=case["master"], state=s["state"])
        s["opt"].step(s["grads"])
        return _adamw_outputs(s, s["opt"].moments() if case["bits"] == 8 else (s["state"]["m"], s["state"]["v"]))
    act = None if case["act"] == "none" else case["act"]
    if op == "linear":
        return trw.linear_forward(s["x"], s["w"], s["bias"], act, s["residual"])
    y, z = trw.linear_forward(s["x"], s["w"], s["bias"], act, s["residual"], save=True)
    dx, dw, db = trw.linear_backward(s["x"], s["w"], z, s["dy"], act, need_db=case["bias"])
    return {"y": y, "dx": dx, "dw": dw, "db": db}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_moe(state) if op == "moe" else _plain_adamw(state) if op == "adamw" else _plain_linear(state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    e = {"f32": 4, "bf16": 2, "f16": 2}
    if case["op"] == "adamw":
        n, p = sum(_sizes(case)), e[case["dtype"]]
        moments = 16 if case["bits"] == 32 else 4 + 4 / BLOCK + 8   # (8 bits: and their values written)
        # with master weights a parameter is only written
        return {"bytes": n * (e[case["grad"]] + (8 + p if case["master"] else 2 * p) + moments), "flops": 16 * n}
    rows, cols, t = case["rows"], case["cols"], case["tokens"]
    if case["op"] == "moe":
        experts, top = case["experts"], case["top"]
        read = experts * (1 - (1 - top / experts) ** t)   # expected number of different experts
        return {"bytes": 2 * (read * 3 * rows * cols + experts * cols + 2 * t * cols),
                "flops": 2 * t * cols * (3 * top * rows + experts)}
    out = t * rows * (2 if case["residual"] else 1) + (rows if case["bias"] else 0)
    read = rows * cols + t * cols
    if case["op"] == "linear":
        return {"bytes": 2 * (read + out), "flops": 2 * t * rows * cols}
    return {"bytes": 2 * (2 * read + out + t * rows), "flops": 6 * t * rows * cols}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(s)
    if case["op"] == "moe":
        return _exact_moe(s)
    x, w = s["x"].double().requires_grad_(True), s["w"].double().requires_grad_(True)
    b = s["bias"].double().requires_grad_(True) if case["bias"] else None
    y = _exact_act(torch.addmm(b, x, w.t()) if case["bias"] else torch.mm(x, w.t()), case["act"])
    if case["residual"]:
        y = y + s["residual"].double()
    if case["op"] == "linear":
        return y.detach()
    grads = torch.autograd.grad(y, [x, w] + ([b] if case["bias"] else []), s["dy"].double())
    return {"y": y.detach(), "dx": grads[0], "dw": grads[1], "db": grads[2] if case["bias"] else None}


def _exact_act(z, act):
    if act == "none":
        return z
    if act == "silu":
        return z * torch.special.expit(z)
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0))
    # (1 + tanh(a)) / 2 = 1 / (1 + exp(-2 a))
    return z * torch.special.expit(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))


def _exact_moe(s):
    case, x = s["case"], s["x"].double()
    logits = (x[:, None, :] * s["wr"].double()).sum(2)
    ids = torch.empty(case["tokens"], case["top"], dtype=torch.int32, device="cuda")
    left = logits.clone()
    for j in range(case["top"]):   # the largest, the lowest index where several are
        best = left.max(1, keepdim=True).values
        ids[:, j] = (left == best).int().argmax(1)
        left.scatter_(1, ids[:, j:j + 1].long(), -math.inf)
    chosen = logits.gather(1, ids.long())
    weights = torch.softmax(chosen, 1) if case["normalize"] else torch.softmax(logits, 1).gather(1, ids.long())
    y = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        w = (weights * (ids == e)).sum(1, keepdim=True)
        at = (ids == e).any(1).nonzero().view(-1)
        if at.numel():
            h = _exact_act(x[at] @ s["wg"][e].double().t(), case["act"]) * (x[at] @ s["wu"][e].double().t())
            y[at] += w[at] * (h @ s["wd"][e].double().t())
    return {"y": y, "ids": ids, "weights": weights}


def _power(exponents):
    """2^exponents, exactly."""
    powers = torch.tensor([math.ldexp(1.0, k) for k in range(-150, 151)], dtype=torch.float64, device="cuda")
    return powers[exponents + 150]


def _coded(values, b, table, top):
    """The nearest of the table's values times 2^(b - top), ties to the even code; the table in order of its codes."""
    scale = _power(b - top)
    wanted = values.abs() / scale
    high = torch.searchsorted(table, wanted.contiguous()).clamp(1, table.numel() - 1)
    low = high - 1
    up, down = table[high] - wanted, wanted - table[low]
    code = torch.where((up < down) | ((up == down) & (high % 2 == 0)), high, low)
    return code, scale


def _exact_adamw(s):
    case, state, sizes = s["case"], s["state"], s["sizes"]
    (b1, b2), t = BETAS, 100
    tables = {"m": [k * 2.0 ** -9 if k < 8 else (8 + k % 8) * 2.0 ** (k // 8 - 10) for k in range(127)],
              "v": [k * 2.0 ** -17 if k < 8 else (8 + k % 8) * 2.0 ** (k // 8 - 18) for k in range(248)]}
    g = torch.cat([torch.cat([x, x.new_zeros(-x.numel() % BLOCK)]) for x in s["grads"]])
    real = torch.cat([torch.arange(-(-n // BLOCK) * BLOCK, device="cuda") < n for n in sizes])
    old, new = {"m": state["m"], "v": state["v"]}, {}
    if case["bits"] == 8:
        count = g.numel()
        for k, top in (("m", 134), ("v", 141)):
            table = torch.tensor(tables[k], dtype=torch.float64, device="cuda")
            code, b = old[k][:count].long(), old[k][count:].long().repeat_interleave(BLOCK)
            sign = torch.where(code > 127, -1.0, 1.0) if k == "m" else 1.0
            old[k] = sign * table[code % 128 if k == "m" else code] * _power(b - top)
    new["m"] = b1 * old["m"].double() + (1 - b1) * g.double()
    new["v"] = b2 * old["v"].double() + (1 - b2) * g.double() ** 2
    rise = (new["m"] / (1 - b1 ** t)) / ((new["v"] / (1 - b2 ** t)).sqrt() + EPS)
    if case["master"]:
        full = state["master"].double()
    else:
        full = torch.zeros_like(rise)
        full[real] = s["flat"].double()
    full = full - LR * DECAY * full - LR * rise
    if case["bits"] == 8:
        # codes are those of moments that are defined by 32-bit steps
        g, old = g.float(), {k: v.float() for k, v in old.items()}
        new = {"m": (old["m"] * b1 + g * (1 - b1)).double(), "v": (old["v"] * b2 + g.square() * (1 - b2)).double()}
        for k, top in (("m", 134), ("v", 141)):
            table = torch.tensor(tables[k], dtype=torch.float64, device="cuda")
            size = new[k].abs()
            b = torch.frexp(size.view(-1, BLOCK).max(1).values).exponent.long() + 126
            b = b.clamp(min=15).repeat_interleave(BLOCK)
            code, scale = _coded(new[k], b, table, top)
            if k == "v":
                code = torch.where((code == 0) & (size > 0), 1, code)
            new[k] = torch.copysign(table[code] * scale, new[k])
    return {"params": full[real], "master": full if case["master"] else None, **new}
