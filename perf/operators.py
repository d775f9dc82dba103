"""Cases of the router's balance loss and of the experts' 4-bit (MX) matrices: what is timed, on which inputs, and
what it has to compute.

Three paths, each as a program that trains or serves a mixture of experts calls it:

* balance: the auxiliary losses of a router with its per-expert counts, and the gradient of its logits (losses and
  gates together): a forward and a backward call of a training step;
* quant: rows to microscaled 4-bit floating point (e2m1 codes, one e8m0 scale per 32 values) and back;
* up, down, dense: a product of two such matrices. up is the experts' gate and up rows with SwiGLU, on tokens
  gathered by the router's choice; down is the experts' down rows, times the gates; dense has one matrix.

With `own` false `run` computes them with elementary torch operations; with `own` true it calls the library.
"""
import math

import torch

own = False

BLOCK = 32  # values per scale
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # a small model's router on a short ragged batch: latency
        {"name": "balance_t37_e16", "kind": "balance", "T": 37, "E": 16, "k": 2, "renorm": True, "mask": True, "drop": False},
        # one prefill-sized chunk, 512 experts
        {"name": "balance_t8192_e512", "kind": "balance", "T": 8192, "E": 512, "k": 10, "renorm": True, "mask": False, "drop": False},
        # a training batch with padding, experts out of use, gates from the full softmax
        {"name": "balance_t65521_e512", "kind": "balance", "T": 65521, "E": 512, "k": 10, "renorm": False, "mask": True, "drop": True},
        # one token's hidden state
        {"name": "quant_1x2048", "kind": "quant", "rows": 1, "cols": 2048, "type": "bf16"},
        # the experts' hidden rows of a chunk, fp16, an odd count
        {"name": "quant_20483x768", "kind": "quant", "rows": 20483, "cols": 768, "type": "fp16"},
        # the gate and up rows of 64 experts, from fp32 weights
        {"name": "quant_98304x2048", "kind": "quant", "rows": 98304, "cols": 2048, "type": "fp32"},
        # one decoded token: ten experts and the shared one
        {"name": "up_t1", "kind": "up", "T": 1, "d": 2048, "f": 768, "E": 512, "k": 10},
        {"name": "down_t3", "kind": "down", "T": 3, "d": 2048, "f": 768, "E": 512, "k": 10},
        # a prefill chunk
        {"name": "up_t8192", "kind": "up", "T": 8192, "d": 2048, "f": 768, "E": 512, "k": 10},
        {"name": "down_t8192", "kind": "down", "T": 8192, "d": 2048, "f": 768, "E": 512, "k": 10},
        # few experts with many rows each, an odd number of tokens: bound by the tensor cores
        {"name": "up_t7919_e16", "kind": "up", "T": 7919, "d": 2048, "f": 1536, "E": 16, "k": 2},
        # one matrix, many rows (a shared expert's gate and up rows alone)
        {"name": "dense_8190x1536", "kind": "dense", "rows": 8190, "n": 1536, "cols": 2048},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["balance", "quant", "up", "down", "dense"])
    if kind == "balance":
        E = _log(rng, 8, 512)
        return {"kind": kind, "T": _log(rng, 1, 65521), "E": E, "k": rng.randint(1, min(E, 12)),
                "renorm": rng.random() < 0.5, "mask": rng.random() < 0.5, "drop": rng.random() < 0.5}
    if kind == "quant":
        return {"kind": kind, "rows": _log(rng, 1, 98304), "cols": 32 * _log(rng, 1, 64),
                "type": rng.choice(sorted(TYPES))}
    if kind == "dense":
        return {"kind": kind, "rows": _log(rng, 1, 8192), "n": 16 * _log(rng, 1, 128), "cols": 32 * _log(rng, 1, 64)}
    E = _log(rng, 8, 512)
    return {"kind": kind, "T": _log(rng, 1, 8192), "d": 128 * rng.randint(1, 16), "f": 64 * rng.randint(1, 12), "E": E,
            "k": rng.randint(1, min(E, 10))}


def work(case):
    kind = case["kind"]
    if kind == "balance":
        T, E, k = case["T"], case["E"], case["k"]
        # logits, choices, gates, gates' gradients and mask in; the logits' gradient, counts and mean probabilities out
        return {"bytes": 8 * T * E + 12 * T * k + T + 8 * E, "flops": 12 * T * E}
    if kind == "quant":
        n, size = case["rows"] * case["cols"], 4 if case["type"] == "fp32" else 2
        # values in; codes, scales and the values that they stand for out
        return {"bytes": 2 * n * size + n // 2 + n // BLOCK, "flops": 4 * n}
    if kind == "dense":
        rows, n, cols = case["rows"], case["n"], case["cols"]
        return {"bytes": 2 * rows * cols + n * cols * 17 // 32 + 2 * rows * n, "flops": 2 * rows * n * cols}
    T, d, f, E, k = (case[x] for x in ("T", "d", "f", "E", "k"))
    rows = T * (k + 1)  # the shared expert takes every token
    used = E * (1 - (1 - k / E) ** T) + 1  # experts with a token, expected
    if kind == "up":
        return {"bytes": int(2 * T * d + used * 2 * f * d * 17 / 32 + 2 * rows * f), "flops": 4 * rows * f * d}
    return {"bytes": int(2 * rows * f + used * f * d * 17 / 32 + 4 * rows * d), "flops": 2 * rows * f * d}


# ---------------------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _top(scores, k):
    """The k largest of each row in descending order, ties to the lower index."""
    v, i = torch.sort(scores, dim=1, descending=True, stable=True)
    return v[:, :k].contiguous(), i[:, :k].to(torch.int32).contiguous()


def _pitch(cols):
    return (cols // BLOCK + 15) // 16 * 16  # bytes of one row of scales


def _weights(g, slots, rows, cols):
    """A pool of `slots` matrices of normal weights (deviation cols^-1/2), as codes and scales."""
    codes = torch.empty(slots, rows, cols // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(slots, rows, _pitch(cols), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // (rows * cols))
    for s in range(0, slots, step):
        n = min(step, slots - s)
        q, e = _levels(_randn(g, n, rows, cols) * cols ** -0.5)
        c = q.reshape(n, rows, cols // 2, 2)
        codes[s:s + n] = c[..., 0] | (c[..., 1] << 4)
        scales[s:s + n, :, :cols // BLOCK] = e
    return codes, scales


_context = None


def _library():
    """The package's binding and one context."""
    global _context
    from bit_expert_ffn_router_b200 import moe
    if _context is None:
        _context = moe.Context(torch.cuda.current_device())
    return moe, _context


def prepare(case, seed):
    g = _gen(seed)
    kind = case["kind"]
    s = {"case": case, "kind": kind}
    if kind == "balance":
        T, E, k = case["T"], case["E"], case["k"]
        logits = _randn(g, T, E) * 1.5 + _randn(g, E)
        if case["drop"]:  # experts out of use, and a few tokens that may use none
            logits[:, torch.rand(E, generator=g, device="cuda") < 0.1] = -math.inf
            logits[torch.rand(T, generator=g, device="cuda") < 0.01] = -math.inf
        v, idx = _top(logits, k)
        ref = v if case["renorm"] else logits
        top = ref.amax(1, keepdim=True).clamp_min(-1e30)
        gate = torch.exp(v - top) / torch.exp(ref - top).sum(1, keepdim=True).clamp_min(1e-30)
        s |= {"logits": logits, "idx": idx, "gate": gate,
              "mask": (torch.rand(T, generator=g, device="cuda") < 0.8).to(torch.uint8) if case["mask"] else None,
              "d_loss": torch.tensor([0.01, 0.001], device="cuda"),
              "d_gate": _randn(g, T, k) * (0.01 / T)}
        if own:
            moe, _ = _library()
            cfg = moe.LayerCfg(d=256, f=128, E=E, k=k, renorm=int(case["renorm"]))
            s |= {"cfg": cfg, "ws": moe.balance_workspace(cfg), "stats": torch.empty(4, device="cuda"),
                  "counts": torch.empty(E, dtype=torch.int32, device="cuda"), "prob": torch.empty(E, device="cuda"),
                  "d_logits": torch.empty(T, E, device="cuda")}
        return s
    if kind == "quant":
        rows, cols, t = case["rows"], case["cols"], TYPES[case["type"]]
        # rows of different size, a few large values, some blocks of zeros
        x = _randn(g, rows, cols) * torch.exp(_randn(g, rows, 1))
        x.view(rows, cols // BLOCK, BLOCK)[torch.rand(rows, cols // BLOCK, generator=g, device="cuda") < 0.01] = 0
        s |= {"x": x.to(t)}
        if own:
            moe, _ = _library()
            s |= {"codes": moe.mx4_buffers(rows, cols), "values": torch.empty(rows, cols, dtype=t, device="cuda")}
        return s
    if kind == "dense":
        rows, n, cols = case["rows"], case["n"], case["cols"]
        codes, scales = _weights(g, 1, n, cols)
        s |= {"x": _randn(g, rows, cols).to(torch.bfloat16), "w": codes, "w_scales": scales, "rows": rows}
        if own:
            moe, _ = _library()
            s |= {"matrix": moe.Mx4Matrix(codes, scales, cols), "codes": moe.mx4_buffers(rows, cols),
                  "out": torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")}
        return s
    T, d, f, E, k = (case[x] for x in ("T", "d", "f", "E", "k"))
    n, cols = (2 * f, d) if kind == "up" else (d, f)
    codes, scales = _weights(g, E + 1, n, cols)
    # the experts lie in the pool in any order; one slot holds the shared expert
    slots = torch.randperm(E + 1, generator=g, device="cuda")
    top, idx = _top(_randn(g, T, E) + 0.3 * _randn(g, E), k)
    gate = torch.exp(top - top[:, :1])
    gate /= gate.sum(1, keepdim=True)
    order = torch.argsort(idx.reshape(-1), stable=True)  # sorted by expert, then token, then rank
    counts = torch.bincount(idx.reshape(-1), minlength=E).tolist()
    slot_of = slots[:E].to(torch.int32).contiguous()
    rows = T * (k + 1)
    x = _randn(g, T, d) if kind == "up" else _randn(g, rows, f) * 0.3
    s |= {"x": x.to(torch.bfloat16), "w": codes, "w_scales": scales, "counts": counts, "token": order // k,
          "pair_gate": gate.reshape(-1)[order], "slots": slots.tolist(), "rows": rows}
    if own:
        moe, ctx = _library()
        cfg = moe.LayerCfg(d=256, f=128, E=E, k=k)  # the grouping goes by E and k alone
        ws = moe.workspace(cfg, T)
        s |= {"ws": ws, "keep": (idx, gate, slot_of), "grouping": ctx.group_tokens(cfg, idx, gate, T, slot_of, E + 1, ws),
              "matrix": moe.Mx4Matrix(codes, scales, cols), "codes": moe.mx4_buffers(x.shape[0], cols),
              "out": torch.empty(rows, f if kind == "up" else d, device="cuda",
                                 dtype=torch.bfloat16 if kind == "up" else torch.float32)}
    return s


# ---------------------------------------------------------------------------------------------------- plain form

_tables = {}


def _table(name):
    if name not in _tables:
        if name == "e2m1":  # code -> value
            v = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
            v += [-a for a in v]
        else:  # e8m0 byte -> scale, exact in 32 bits
            v = [2.0 ** (i - 127) for i in range(255)] + [math.nan]
        _tables[name] = torch.tensor(v, dtype=torch.float32, device="cuda")
    return _tables[name]


def _levels(x):
    """[..., K] -> e2m1 codes [..., K] and e8m0 scales [..., K/32] (uint8)."""
    v = x.float().reshape(*x.shape[:-1], x.shape[-1] // BLOCK, BLOCK)
    top = v.abs().amax(-1)
    e = torch.where(top > 0, torch.frexp(top)[1] - 3, -127).clamp(-127, 127)
    bad = ~(top < math.inf)
    a = v * _table("e8m0")[(127 - e).long()].unsqueeze(-1)  # times 2^-e: exact
    m = a.abs()
    q = torch.where(m < 2, torch.round(m * 2), torch.where(m < 4, torch.round(m) + 2, torch.round(m * 0.5) + 4))
    q = torch.nan_to_num(q, nan=0.0, posinf=7.0).clamp_max(7).to(torch.uint8) | (torch.signbit(a).to(torch.uint8) << 3)
    return q.reshape(x.shape), torch.where(bad, 255, e + 127).to(torch.uint8)


def _values(q, e):
    """The 32-bit values that codes and scales stand for."""
    v = _table("e2m1")[q.long()].reshape(*e.shape, BLOCK) * _table("e8m0")[e.long()].unsqueeze(-1)
    return v.reshape(q.shape)


def _unpack(codes, scales):
    q = torch.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], codes.shape[-1] * 2)
    return _values(q, scales[..., :q.shape[-1] // BLOCK])


def _balance(s):
    case, logits, k = s["case"], s["logits"], s["case"]["k"]
    T, E = logits.shape
    keep = logits.amax(1) != -math.inf
    if s["mask"] is not None:
        keep &= s["mask"] != 0
    keep = keep.unsqueeze(1)
    l = torch.where(keep, logits, 0.0)
    top = l.amax(1, keepdim=True)
    p = torch.exp(l - top)
    total = p.sum(1, keepdim=True)
    lse = torch.where(keep, top + torch.log(total), 0.0)
    p = torch.where(keep, p / total, 0.0)
    idx = s["idx"].long()
    counts = torch.zeros(E, dtype=torch.int32, device="cuda")
    counts.scatter_add_(0, idx.reshape(-1), keep.expand(T, k).reshape(-1).to(torch.int32))
    n = keep.sum().double()
    m = n.clamp_min(1)
    prob = p.sum(0, dtype=torch.float64) / m
    load = counts.double() * (E / k) / m
    stats = torch.stack(((load * prob).sum(), (lse.double() ** 2).sum() / m, n, load.max())).float()
    load32 = load.float()
    d = p * (s["d_loss"][0] / m.float() * (load32 - (p * load32).sum(1, keepdim=True))
             + s["d_loss"][1] * 2 / m.float() * lse)
    gate, dg = s["gate"], s["d_gate"]
    gdg = gate * dg
    if case["renorm"]:
        gdg = gdg - gate * gdg.sum(1, keepdim=True)
    else:
        d = d - p * gdg.sum(1, keepdim=True)
    d = d.scatter_add(1, idx, torch.where(keep, gdg, 0.0))
    return {"stats": stats, "counts": counts, "prob": prob.float(), "d_logits": d}


def _groups(s):
    """(slot, first row, rows) of every expert that has rows, the shared expert last."""
    row = 0
    for e, n in enumerate(s["counts"]):
        if n:
            yield s["slots"][e], row, n
        row += n
    T = s["rows"] - row
    yield s["slots"][-1], row, T


def _plain(s):
    kind = s["kind"]
    if kind == "balance":
        return _balance(s)
    x = _values(*_levels(s["x"]))
    if kind == "quant":
        return x.to(s["x"].dtype)
    if kind == "dense":
        return (x @ _unpack(s["w"][0], s["w_scales"][0]).T).to(torch.bfloat16)
    pairs = s["token"].numel()
    out = []
    for slot, row, n in _groups(s):
        w = _unpack(s["w"][slot], s["w_scales"][slot])
        if kind == "up":
            a = x if row == pairs else x[s["token"][row:row + n]]
            gu = a @ w.T
            gate, up = gu[:, 0::2], gu[:, 1::2]
            out.append((gate / (1 + torch.exp(-gate)) * up).to(torch.bfloat16))
        else:
            z = x[row:row + n] @ w.T
            out.append(z if row == pairs else z * s["pair_gate"][row:row + n].unsqueeze(1))
    return torch.cat(out)


# ---------------------------------------------------------------------------------------------------- the pass

def run(state):
    if not own:
        return _plain(state)
    moe, ctx = _library()
    kind = state["kind"]
    if kind == "balance":
        s, cfg, T = state, state["cfg"], state["case"]["T"]
        ctx.balance_loss(cfg, s["logits"], s["idx"], s["mask"], T, s["stats"], s["counts"], s["prob"], s["ws"])
        ctx.balance_loss_backward(cfg, s["logits"], s["idx"], s["gate"], s["mask"], T, s["stats"], s["counts"],
                                  s["d_loss"], s["d_gate"], s["d_logits"])
        return {"stats": s["stats"], "counts": s["counts"], "prob": s["prob"], "d_logits": s["d_logits"]}
    codes, scales = state["codes"]
    ctx.mx4_quantize(state["x"], codes, scales)
    if kind == "quant":
        ctx.mx4_dequantize(codes, scales, state["values"])
        return state["values"]
    if kind == "dense":
        ctx.mx4_product(codes, scales, state["matrix"], state["out"])
    elif kind == "up":
        ctx.mx4_product(codes, scales, state["matrix"], state["out"], grouping=state["grouping"],
                        shared_slot=state["slots"][-1], gather=True, swiglu=True)
    else:
        ctx.mx4_product(codes, scales, state["matrix"], state["out"], grouping=state["grouping"],
                        shared_slot=state["slots"][-1], gate=True)
    return state["out"]


# ---------------------------------------------------------------------------------------------------- 64 bits

def _exact_quant(x):
    """Rounds [..., K] to the format by comparing with the middles between its levels, in 64 bits."""
    v = x.double().unflatten(-1, (-1, BLOCK))
    big = v.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(big.clamp_min(2.0 ** -160)))
    e = torch.where(torch.exp2(e) > big, e - 1, torch.where(torch.exp2(e + 1) <= big, e + 1, e))
    scale = torch.exp2((e - 2).clamp(-127, 127))
    a = v.abs() / scale
    r = torch.zeros_like(a)
    # a middle goes to the level whose last bit is 0
    for middle, step, up in ((0.25, .5, False), (0.75, .5, True), (1.25, .5, False), (1.75, .5, True), (2.5, 1., False),
                             (3.5, 1., True), (5., 2., False)):
        r += step * ((a >= middle) if up else (a > middle))
    return (torch.copysign(r, v) * scale).flatten(-2)


def _exact_weights(codes, scales, cols):
    out = torch.empty(codes.shape[0], cols, dtype=torch.float64, device="cuda")
    for half in range(2):
        c = ((codes >> (4 * half)) & 15).int()
        m, ex = c & 1, (c >> 1) & 3
        mag = torch.where(ex == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(ex.double() - 1))
        out[:, half::2] = torch.where(c >= 8, -mag, mag)
    return out * torch.exp2(scales[:, :cols // BLOCK].double() - 127).repeat_interleave(BLOCK, dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "balance":
        return _exact_balance(s)
    if kind == "quant":
        step = max(1, (1 << 24) // case["cols"])
        return torch.cat([_exact_quant(c) for c in s["x"].split(step)])
    x = _exact_quant(s["x"])
    if kind == "dense":
        return x @ _exact_weights(s["w"][0], s["w_scales"][0], case["cols"]).T
    cols = case["d"] if kind == "up" else case["f"]
    res = torch.empty(s["rows"], case["f"] if kind == "up" else case["d"], dtype=torch.float64, device="cuda")
    pairs = s["token"].numel()
    first = 0
    for e, n in enumerate(s["counts"] + [s["rows"] - pairs]):
        if not n:
            continue
        slot, rows = s["slots"][e], slice(first, first + n)
        first += n
        w = _exact_weights(s["w"][slot], s["w_scales"][slot], cols)
        if kind == "up":
            a = x[s["token"][rows]] if e < case["E"] else x
            res[rows] = torch.nn.functional.silu(a @ w[0::2].T) * (a @ w[1::2].T)
        else:
            res[rows] = x[rows] @ w.T
            if e < case["E"]:
                res[rows] *= s["pair_gate"][rows].double()[:, None]
    return res


def _exact_balance(s):
    """The losses as functions of the logits in 64 bits, and their gradient by automatic differentiation."""
    case = s["case"]
    E, k = case["E"], case["k"]
    use = (s["logits"] > -math.inf).any(1) | s["logits"].isnan().any(1)
    if s["mask"] is not None:
        use &= s["mask"].bool()
    rows = use.nonzero()[:, 0]
    n = rows.numel()
    full = torch.zeros(s["logits"].shape, dtype=torch.float64, device="cuda")
    counts = torch.bincount(s["idx"][rows].reshape(-1).long(), minlength=E)
    if n == 0:
        return {"stats": torch.zeros(4, dtype=torch.float64, device="cuda"), "counts": counts.int(),
                "prob": full[0] * 0, "d_logits": full}
    with torch.enable_grad():
        l = s["logits"][rows].double().requires_grad_()
        prob = torch.softmax(l, 1).mean(0)
        load = counts.double() * E / (k * n)
        balance, z = (load * prob).sum(), (torch.logsumexp(l, 1) ** 2).mean()
        idx = s["idx"][rows].long()
        gate = torch.softmax(l.gather(1, idx), 1) if case["renorm"] else torch.softmax(l, 1).gather(1, idx)
        dl = s["d_loss"].double()
        total = dl[0] * balance + dl[1] * z + (gate * s["d_gate"][rows].double()).sum()
        grad, = torch.autograd.grad(total, l)
    full[rows] = grad
    stats = torch.stack((balance.detach(), z.detach(), torch.tensor(float(n), dtype=torch.float64, device="cuda"), load.max()))
    return {"stats": stats, "counts": counts.int(), "prob": prob.detach(), "d_logits": full}
