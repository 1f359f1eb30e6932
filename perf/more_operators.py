"""What is measured of the expert block's operators: the gated feed-forward of
the experts, 8-bit rows on the way to them, and dropout on the way back.

  ffn        y = (act(x Wg') * (x Wu')) Wo' of each expert's rows: training
             (the pre-activations and the product kept) or serving (y alone);
  ffn_grad   its gradients of x and both weights, from what the forward kept;
  norm8      y = x + block, and the root-mean-square norm of y times a weight
             in 8 bits with one scale per row, read back as the receiving
             process of an exchange does;
  dispatch8  such rows copied into expert order as values of the model's type;
  dropout    elements kept where a counter-based random number says so, scaled,
             with the residual added or, as in the backward pass, alone.

`run` takes the plain torch form where `own` is false and the library's entry
points where it is true.  `exact` gives the outputs in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
NORM_EPS = 1e-6


def listed():
    return [
        # serving: eight samples, two of eight experts, 16 rows in all: latency
        {"name": "ffn_16x512_bf16", "op": "ffn", "tokens": 8, "topk": 2, "experts": 8,
         "capacity": 0, "dim": 512, "hidden": 1024, "kind": "bf16", "act": "silu",
         "train": False, "absent": 0.0},
        # serving a wide block: every weight is read for one or two rows
        {"name": "ffn_64x3328_bf16", "op": "ffn", "tokens": 32, "topk": 2, "experts": 32,
         "capacity": 0, "dim": 3328, "hidden": 1664, "kind": "bf16", "act": "silu",
         "train": False, "absent": 0.0},
        # one dense block on the interaction's output width (odd)
        {"name": "ffn_4096x479_f32", "op": "ffn", "tokens": 4096, "topk": 1, "experts": 1,
         "capacity": 0, "dim": 479, "hidden": 1000, "kind": "f32", "act": "gelu",
         "train": True, "absent": 0.0},
        # the concatenated pooled rows of 26 tables (26 * 128 wide), ragged groups
        {"name": "ffn_32768x3328_bf16", "op": "ffn", "tokens": 16_384, "topk": 2, "experts": 16,
         "capacity": 0, "dim": 3328, "hidden": 1664, "kind": "bf16", "act": "silu",
         "train": True, "absent": 0.02},
        # experts at a fixed capacity, odd width
        {"name": "ffn_grad_10240x479_f32", "op": "ffn_grad", "tokens": 4096, "topk": 2,
         "experts": 8, "capacity": 1280, "dim": 479, "hidden": 640, "kind": "f32",
         "act": "silu", "absent": 0.0},
        {"name": "ffn_grad_32768x3328_bf16", "op": "ffn_grad", "tokens": 16_384, "topk": 2,
         "experts": 16, "capacity": 0, "dim": 3328, "hidden": 1664, "kind": "bf16",
         "act": "silu", "absent": 0.02},
        # a small batch of the interaction's output before the exchange
        {"name": "norm8_256x479_f32", "op": "norm8", "rows": 256, "dim": 479, "kind": "f32"},
        {"name": "norm8_65536x3328_bf16", "op": "norm8", "rows": 65_536, "dim": 3328,
         "kind": "bf16"},
        # a serving batch: latency
        {"name": "dispatch8_64x512_bf16", "op": "dispatch8", "tokens": 64, "topk": 2,
         "experts": 8, "capacity": 0, "dim": 512, "kind": "bf16", "absent": 0.0},
        {"name": "dispatch8_32768x3328_bf16", "op": "dispatch8", "tokens": 32_768, "topk": 2,
         "experts": 64, "capacity": 0, "dim": 3328, "kind": "bf16", "absent": 0.02},
        # the gradient of a small tower layer's dropout
        {"name": "dropout_1024x479_f32", "op": "dropout", "numel": 1024 * 479, "kind": "f32",
         "p": 0.1, "residual": False},
        # a wide block's output on the way to the residual stream
        {"name": "dropout_65536x3328_bf16", "op": "dropout", "numel": 65_536 * 3328,
         "kind": "bf16", "p": 0.2, "residual": True},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def width():
        return rng.choice([64, 128, 351, 479, 512, 1000, 1664, 3328, log(17, 4000)])

    op = rng.choice(["ffn", "ffn", "ffn_grad", "ffn_grad", "norm8", "dispatch8", "dropout"])
    kind = rng.choice(["f32", "bf16", "bf16", "f16"])
    if op == "dropout":
        return {"op": op, "numel": log(500, 65_536 * 3328 // 2), "kind": kind,
                "p": rng.choice([0.05, 0.1, 0.5, round(rng.uniform(0.0, 0.9), 3)]),
                "residual": rng.random() < 0.5}
    dim = width()
    if op == "norm8":
        most = 65_536 * 3328 // 2
        return {"op": op, "rows": max(1, min(log(1, 65_536), most // dim)), "dim": dim,
                "kind": kind}
    if op == "dispatch8":
        e = rng.choice([2, 4, 8, 16, 32, 64, 100, 256])
        k = rng.randint(1, min(e, 8))
        n = max(1, min(log(1, 65_536), 32_768 * 2 * 3328 // 2 // (k * dim)))
        cap = 0 if rng.random() < 0.6 else max(1, int(n * k / e * rng.uniform(0.8, 1.5)))
        return {"op": op, "tokens": n, "topk": k, "experts": e, "capacity": cap, "dim": dim,
                "kind": kind, "absent": rng.choice([0.0, 0.02, 0.3])}
    e = rng.choice([1, 2, 4, 8, 16, 32])
    k = rng.randint(1, min(e, 4))
    hidden = rng.choice([dim // 2 + 8, dim, dim * 3 // 2 + 1, width()])
    while e * dim * hidden > 32 * 3328 * 1664:
        e //= 2
        k = min(k, e)
    most = 32_768 * 3328 * 1664 // 2
    n = max(1, min(log(1, 32_768), most // (k * dim * hidden)))
    cap = 0 if e == 1 or rng.random() < 0.6 else max(1, int(n * k / e * rng.uniform(0.8, 1.5)))
    case = {"op": op, "tokens": n, "topk": k, "experts": e, "capacity": cap, "dim": dim,
            "hidden": hidden, "kind": kind, "act": rng.choice(["silu", "gelu", "relu", "sigmoid"]),
            "absent": 0.0 if e == 1 else rng.choice([0.0, 0.02, 0.3])}
    if op == "ffn":
        case["train"] = rng.random() < 0.5
    return case


# ---------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _choices(case, g):
    """Expert ids [tokens, topk]; some experts are liked better than others, and a
    padded sample has none (-2)."""
    n, k, e = case["tokens"], case["topk"], case["experts"]
    logits = torch.randn(n, e, generator=g, device=DEV) + torch.randn(e, generator=g, device=DEV)
    ids = torch.topk(logits, k, dim=1).indices
    gone = torch.rand(n, 1, generator=g, device=DEV) < case["absent"]
    return torch.where(gone, -2, ids)


def _buffer_rows(case):
    return case["experts"] * case["capacity"] if case["capacity"] else \
        case["tokens"] * case["topk"]


def _groups(case, g):
    """Each expert's rows of the expert-ordered buffer, as (first, count) pairs."""
    ids = _choices(case, g)
    counts = [int(c) for c in torch.bincount(ids[ids >= 0], minlength=case["experts"]).tolist()]
    c = case["capacity"]
    if c:
        return [(i * c, min(n, c)) for i, n in enumerate(counts)]
    return [(sum(counts[:i]), n) for i, n in enumerate(counts)]


def _act(case, v):
    """The activation and its derivative."""
    if case["act"] == "relu":
        on = v > 0
        return torch.where(on, v, 0.0), on.to(v.dtype)
    if case["act"] == "gelu":
        half = 0.5 * torch.erfc(v * -math.sqrt(0.5))
        return v * half, half + v * torch.exp(-0.5 * v * v) * (1 / math.sqrt(2 * math.pi))
    s = 1 / (1 + torch.exp(-v))
    slope = 1 / (1 + torch.exp(v)) * s
    return (s, slope) if case["act"] == "sigmoid" else (v * s, s + v * slope)


def _ffn_inputs(case, g):
    e, d, f, t = case["experts"], case["dim"], case["hidden"], DTYPES[case["kind"]]
    groups = _groups(case, g)
    m = _buffer_rows(case)
    x = torch.randn(m, d, generator=g, device=DEV).to(t)
    w_in = (torch.randn(e, 2 * f, d, generator=g, device=DEV) / math.sqrt(d)).to(t)
    w_out = (torch.randn(e, d, f, generator=g, device=DEV) / math.sqrt(f)).to(t)
    if case["op"] == "ffn":
        return groups, x, w_in, w_out, None, None, None
    gu = torch.randn(m, 2 * f, generator=g, device=DEV).to(t)  # normal, as x Wg' and x Wu' are
    a = (_act(case, gu[:, :f].float())[0] * gu[:, f:].float()).to(t)
    dy = torch.randn(m, d, generator=g, device=DEV).to(t)
    return groups, x, w_in, w_out, gu, a, dy


def _norm_inputs(case, g):
    n, d, t = case["rows"], case["dim"], DTYPES[case["kind"]]
    x = torch.randn(n, d, generator=g, device=DEV).to(t)
    block = (torch.randn(n, d, generator=g, device=DEV) * 0.5).to(t)
    return x, block, 1 + 0.1 * torch.randn(d, generator=g, device=DEV)


def _dispatch_inputs(case, g):
    """Rows as another process sent them: codes, scales, and the choices' places."""
    n, k, d = case["tokens"], case["topk"], case["dim"]
    ids = _choices(case, g)
    codes = torch.clamp(torch.randn(n, d, generator=g, device=DEV) * 35, -127, 127).round().to(
        torch.int8)
    scales = (1 + 0.2 * torch.rand(n, generator=g, device=DEV)) / 35
    m = _buffer_rows(case)
    flat = ids.reshape(-1)
    key = torch.where(flat >= 0, flat, case["experts"])
    order = torch.argsort(key, stable=True)
    key = key[order]
    count = torch.bincount(key, minlength=case["experts"] + 1)
    start = torch.cumsum(count, 0) - count
    rank = torch.arange(n * k, device=DEV) - start[key]
    kept, row = key < case["experts"], start[key] + rank
    if case["capacity"]:
        kept, row = kept & (rank < case["capacity"]), key * case["capacity"] + rank
    src = torch.full((m + 1,), -1, dtype=torch.int32, device=DEV)
    src[torch.where(kept, row, m)] = torch.where(kept, order, -1).int()
    pos = torch.empty(n * k, dtype=torch.int32, device=DEV)
    pos[order] = torch.where(kept, row, -1).int()
    return codes, scales, src[:m].contiguous(), pos.reshape(n, k)


def _dropout_inputs(case, g):
    n, t = case["numel"], DTYPES[case["kind"]]
    x = torch.randn(n, generator=g, device=DEV).to(t)
    res = torch.randn(n, generator=g, device=DEV).to(t) if case["residual"] else None
    rng = torch.randint(0, 1 << 62, (2,), generator=g, device=DEV)  # seed and counter
    return x, res, rng


# ---------------------------------------------------------------- prepare

def prepare(case, seed):
    g = _generator(seed)
    s = {"case": case}
    if case["op"] in ("ffn", "ffn_grad"):
        s["groups"], s["x"], s["w_in"], s["w_out"], s["gu"], s["a"], s["dy"] = \
            _ffn_inputs(case, g)
    elif case["op"] == "norm8":
        s["x"], s["block"], s["w"] = _norm_inputs(case, g)
    elif case["op"] == "dispatch8":
        s["codes"], s["scales"], s["src"], s["pos"] = _dispatch_inputs(case, g)
    else:
        s["x"], s["res"], s["rng"] = _dropout_inputs(case, g)
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """The offsets, workspaces and output buffers a program keeps."""
    from recommender_embedding_tables_amd import embtab as eb
    case = s["case"]
    if case["op"] in ("ffn", "ffn_grad"):
        m, e, d, f = s["x"].shape[0], case["experts"], case["dim"], case["hidden"]
        s["code"] = eb.dtype_code(s["x"].dtype)
        s["act"] = {"silu": eb.EMB_ACT_SILU, "gelu": eb.EMB_ACT_GELU, "relu": eb.EMB_ACT_RELU,
                    "sigmoid": eb.EMB_ACT_SIGMOID}[case["act"]]
        ends = [0]
        for _, n in s["groups"]:
            ends.append(ends[-1] + n)
        s["offsets"] = torch.tensor(ends, dtype=torch.int32, device=DEV)
        if e == 1:  # a dense block has no offsets
            s["offsets"] = None
        s["ws_bytes"] = eb.emb_gated_ffn_workspace_bytes(m, e, d, f, s["code"])
        s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device=DEV)
        if case["op"] == "ffn":  # zeros: the rows of no expert are left as they are
            s["y"] = torch.zeros_like(s["x"])
            s["a"] = s["x"].new_zeros(m, f)
            s["gu"] = s["x"].new_zeros(m, 2 * f) if case["train"] else None
        else:
            s["dx"] = torch.zeros_like(s["x"])
            s["dw_in"], s["dw_out"] = torch.empty_like(s["w_in"]), torch.empty_like(s["w_out"])
    elif case["op"] == "norm8":
        n, d = s["x"].shape
        s["y"] = torch.empty_like(s["x"])
        s["codes"] = torch.empty(n, d, dtype=torch.int8, device=DEV)
        s["scales"] = torch.empty(n, device=DEV)
        s["values"] = torch.empty(n, d, dtype=torch.bfloat16, device=DEV)
        s["place"] = torch.arange(n, dtype=torch.int32, device=DEV)  # in the order sent
    elif case["op"] == "dispatch8":
        s["xs"] = torch.empty(s["src"].numel(), case["dim"], dtype=DTYPES[case["kind"]],
                              device=DEV)
    else:
        s["y"] = torch.empty_like(s["x"])


# ---------------------------------------------------------------- run

def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _ffn(s):
    case, t = s["case"], s["x"].dtype
    f, m = case["hidden"], s["x"].shape[0]
    gu = torch.zeros(m, 2 * f, device=DEV)
    a = torch.zeros(m, f, device=DEV)
    y = torch.zeros(m, case["dim"], device=DEV)
    for e, (r, n) in enumerate(s["groups"]):
        if n == 0:
            continue
        gu[r:r + n] = torch.mm(s["x"][r:r + n].float(), s["w_in"][e].float().t())
        a[r:r + n] = _act(case, gu[r:r + n, :f])[0] * gu[r:r + n, f:]
        y[r:r + n] = torch.mm(a[r:r + n], s["w_out"][e].float().t())
    return [gu.to(t), a.to(t), y.to(t)] if case["train"] else [y.to(t)]


def _ffn_grad(s):
    case, t = s["case"], s["x"].dtype
    f = case["hidden"]
    dx = torch.zeros_like(s["x"])
    dw_in, dw_out = torch.zeros_like(s["w_in"]), torch.zeros_like(s["w_out"])
    for e, (r, n) in enumerate(s["groups"]):
        if n == 0:
            continue
        x, a, dy, gu = (s[k][r:r + n].float() for k in ("x", "a", "dy", "gu"))
        dw_out[e] = torch.mm(dy.t(), a).to(t)
        da = torch.mm(dy, s["w_out"][e].float())
        act, slope = _act(case, gu[:, :f])
        dgu = torch.cat([da * gu[:, f:] * slope, da * act], 1)
        dx[r:r + n] = torch.mm(dgu, s["w_in"][e].float()).to(t)
        dw_in[e] = torch.mm(dgu.t(), x).to(t)
    return [dx, dw_in, dw_out]


def _norm8(s):
    y = s["x"].float() + s["block"].float()
    r = torch.rsqrt((y * y).mean(1, keepdim=True) + NORM_EPS)
    h = y * r * s["w"]
    amax = h.abs().amax(1, keepdim=True)
    codes = torch.where(amax > 0, torch.round(h * (127 / amax)), 0.0)
    scale = amax / 127
    values = torch.clamp(codes, -127, 127) * scale
    return [y.to(s["x"].dtype), values.to(torch.bfloat16), scale[:, 0]]


def _dispatch8(s):
    src, k = s["src"], s["case"]["topk"]
    token = torch.clamp(src, min=0).long() // k
    xs = s["codes"][token].float() * s["scales"][token][:, None]
    return [torch.where((src >= 0)[:, None], xs, 0.0).to(DTYPES[s["case"]["kind"]])]


def _mix(v):
    """One SplitMix64 step of 64-bit words."""
    v = v - 7046029254386353131  # the odd number nearest 2^64 over the golden ratio
    v = (v ^ (v >> 30) & (1 << 34) - 1) * -4658895280553007687
    v = (v ^ (v >> 27) & (1 << 37) - 1) * -7723592293110705685
    return v ^ (v >> 31) & (1 << 33) - 1


def _dropout(s):
    n, p = s["case"]["numel"], s["case"]["p"]
    keep = math.floor((1 - p) * 65_536 + 0.5)  # of 2^16 values
    group = s["rng"][1] + torch.arange((n + 3) // 4, device=DEV)
    h = _mix(_mix(s["rng"][0]) ^ group)
    bits = torch.stack([(h >> 16 * j) & 0xFFFF for j in range(4)], 1).reshape(-1)[:n]
    y = torch.where(bits < keep, s["x"].float() * (65_536 / keep if keep else 0.0), 0.0)
    if s["res"] is not None:
        y = y + s["res"].float()
    return [y.to(s["x"].dtype)]


_plain = {"ffn": _ffn, "ffn_grad": _ffn_grad, "norm8": _norm8, "dispatch8": _dispatch8,
          "dropout": _dropout}


def _own_ffn(s):
    from recommender_embedding_tables_amd import embtab as eb
    c = s["case"]
    eb.check(eb.emb_gated_ffn_forward(
        s["x"], s["w_in"], s["w_out"], s["offsets"], s["x"].shape[0], c["experts"], c["capacity"],
        c["dim"], c["hidden"], s["code"], s["act"], s["gu"], s["a"], s["y"], s["ws"],
        s["ws_bytes"]), "gated_ffn")
    return [s["gu"], s["a"], s["y"]] if c["train"] else [s["y"]]


def _own_ffn_grad(s):
    from recommender_embedding_tables_amd import embtab as eb
    c = s["case"]
    eb.check(eb.emb_gated_ffn_backward(
        s["x"], s["gu"], s["a"], s["w_in"], s["w_out"], s["dy"], s["offsets"], s["x"].shape[0],
        c["experts"], c["capacity"], c["dim"], c["hidden"], s["code"], s["act"], s["dx"],
        s["dw_in"], s["dw_out"], s["ws"], s["ws_bytes"]), "gated_ffn_backward")
    return [s["dx"], s["dw_in"], s["dw_out"]]


def _own_norm8(s):
    from recommender_embedding_tables_amd import embtab as eb
    n, d = s["x"].shape
    eb.check(eb.emb_add_norm_int8(s["x"], s["block"], s["w"], n, d, eb.dtype_code(s["x"].dtype),
                                  NORM_EPS, s["y"], s["codes"], s["scales"]), "add_norm_int8")
    eb.check(eb.emb_expert_dispatch_int8(s["codes"], s["scales"], s["place"], s["place"], n, 1, n,
                                         d, eb.EMB_BF16, s["values"]), "expert_dispatch_int8")
    return [s["y"], s["values"], s["scales"]]


def _own_dispatch8(s):
    from recommender_embedding_tables_amd import embtab as eb
    c = s["case"]
    eb.check(eb.emb_expert_dispatch_int8(
        s["codes"], s["scales"], s["pos"], s["src"], c["tokens"], c["topk"], s["src"].numel(),
        c["dim"], eb.dtype_code(s["xs"].dtype), s["xs"]), "expert_dispatch_int8")
    return [s["xs"]]


def _own_dropout(s):
    from recommender_embedding_tables_amd import embtab as eb
    eb.check(eb.emb_dropout(s["x"], s["res"], s["case"]["numel"], eb.dtype_code(s["x"].dtype),
                            s["case"]["p"], s["rng"], s["y"]), "dropout")
    return [s["y"]]


_own = {"ffn": _own_ffn, "ffn_grad": _own_ffn_grad, "norm8": _own_norm8,
        "dispatch8": _own_dispatch8, "dropout": _own_dropout}


# ---------------------------------------------------------------- work

def work(case):
    i = {"f32": 4, "bf16": 2, "f16": 2}[case["kind"]]
    if case["op"] == "dropout":
        n = case["numel"]
        return {"bytes": i * n * (3 if case["residual"] else 2), "flops": 4 * n}
    d = case["dim"]
    if case["op"] == "norm8":
        n = case["rows"]
        return {"bytes": n * d * (3 * i + 4) + 16 * n + 4 * d, "flops": 9 * n * d}
    kept = case["tokens"] * case["topk"] * (1 - case["absent"])
    m = _buffer_rows(case)
    if case["capacity"]:
        kept = min(kept, m)
    if case["op"] == "dispatch8":
        n = case["tokens"]
        return {"bytes": int(n * (d + 4) + m * (i * d + 4) + 4 * n * case["topk"]),
                "flops": int(kept * d)}
    f, e = case["hidden"], case["experts"]
    # experts that get a row when the choices are even
    used = e * -math.expm1(kept * math.log1p(-1 / e)) if e > 1 else 1
    weights = 3 * i * f * d
    if case["op"] == "ffn":
        kept_values = 2 * d + (3 * f if case["train"] else 0)
        return {"bytes": int(i * kept * kept_values + used * weights),
                "flops": int(6 * kept * d * f)}
    return {"bytes": int(i * kept * (3 * d + 3 * f) + (used + e) * weights),
            "flops": int(12 * kept * d * f)}


# ---------------------------------------------------------------- exact

def exact(case, seed):
    g = _generator(seed)
    return {"ffn": _exact_ffn, "ffn_grad": _exact_ffn, "norm8": _exact_norm8,
            "dispatch8": _exact_dispatch8, "dropout": _exact_dropout}[case["op"]](case, g)


def _exact_gate(name, v):
    """The activation of 64-bit values by torch's functions, whose derivative
    automatic differentiation takes."""
    fn = torch.nn.functional
    return {"silu": fn.silu, "gelu": fn.gelu, "relu": fn.relu, "sigmoid": torch.sigmoid}[name](v)


def _exact_ffn(case, g):
    groups, x, w_in, w_out, gu, a, dy = _ffn_inputs(case, g)
    d, f, m = case["dim"], case["hidden"], x.shape[0]
    z = dict(dtype=torch.float64, device=DEV)
    if case["op"] == "ffn":
        pre, prod, y = torch.zeros(m, 2 * f, **z), torch.zeros(m, f, **z), torch.zeros(m, d, **z)
        for e, (r, n) in enumerate(groups):
            mine = slice(r, r + n)
            gate, up = (x[mine].double() @ w_in[e].double().t()).split(f, 1)
            pre[mine, :f], pre[mine, f:] = gate, up
            prod[mine] = _exact_gate(case["act"], gate) * up
            y[mine] = prod[mine] @ w_out[e].double().t()
        return [pre, prod, y] if case["train"] else [y]
    dx = torch.zeros(m, d, **z)
    dw_in, dw_out = torch.zeros(w_in.shape, **z), torch.zeros(w_out.shape, **z)
    for e, (r, n) in enumerate(groups):
        mine = slice(r, r + n)
        # the forward's function of the pre-activations, differentiated
        pre = gu[mine].double().requires_grad_()
        up_grad = dy[mine].double()
        prod = _exact_gate(case["act"], pre[:, :f]) * pre[:, f:]
        dpre, = torch.autograd.grad(prod, pre, up_grad @ w_out[e].double())
        dx[mine] = dpre @ w_in[e].double()
        dw_in[e] = dpre.t() @ x[mine].double()
        dw_out[e] = up_grad.t() @ a[mine].double()  # the product as it was stored
    return [dx, dw_in, dw_out]


def _exact_norm8(case, g):
    x, block, w = _norm_inputs(case, g)
    y = x.double() + block.double()
    h = w.double() * y / torch.sqrt(y.pow(2).sum(1, keepdim=True) / case["dim"] + NORM_EPS)
    step = torch.linalg.vector_norm(h, math.inf, dim=1, keepdim=True) / 127
    return [y, torch.round(h / step) * step, step[:, 0]]


def _exact_dispatch8(case, g):
    codes, scales, src, pos = _dispatch_inputs(case, g)
    values = codes.double() * scales.double()[:, None]
    xs = torch.zeros(src.numel(), case["dim"], dtype=torch.float64, device=DEV)
    for j in range(case["topk"]):  # each token's rows, one choice after another
        on = pos[:, j] >= 0
        xs[pos[on, j].long()] = values[on]
    return [xs]


def _exact_dropout(case, g):
    """The kept elements by the definition, the random words in unsigned arithmetic
    on two 32-bit halves."""
    x, res, rng = _dropout_inputs(case, g)
    seed, counter = (int(v) for v in rng.tolist())
    low = (1 << 32) - 1

    def times(hi, lo, c):  # 64-bit product: 16-bit limbs of the constant, no overflow
        out_lo, out_hi = torch.zeros_like(lo), torch.zeros_like(hi)
        for j in range(4):
            limb = (c >> 16 * j) & 0xFFFF
            part_lo, part_hi = lo * limb, hi * limb  # below 2^48
            if j < 2:
                shifted = (part_lo & ((1 << 48 - 16 * j) - 1)) << 16 * j
                if j == 1:  # bits that the shift would push past 2^63
                    shifted = (part_lo & low >> 16) << 16
                    out_hi = out_hi + (part_lo >> 16)
                    out_hi = out_hi + ((part_hi << 16) & low)
                    out_lo = out_lo + shifted
                else:
                    out_lo = out_lo + (shifted & low)
                    out_hi = out_hi + (shifted >> 32) + part_hi
            else:
                out_hi = out_hi + ((part_lo << 16 * (j - 2)) & low)
        out_hi = out_hi + (out_lo >> 32)
        return out_hi & low, out_lo & low

    def xor_shift(hi, lo, n):
        return hi ^ (hi >> n), lo ^ (((lo >> n) | (hi << 32 - n)) & low)

    def step(hi, lo):
        lo = lo + 0x7F4A7C15
        hi = (hi + 0x9E3779B9 + (lo >> 32)) & low
        hi, lo = xor_shift(hi, lo & low, 30)
        hi, lo = xor_shift(*times(hi, lo, 0xBF58476D1CE4E5B9), 27)
        return xor_shift(*times(hi, lo, 0x94D049BB133111EB), 31)

    def halves(v):
        return v >> 32 & low, v & low

    n = x.numel()
    key = step(*halves(torch.tensor(seed, device=DEV)))
    hi, lo = halves(counter + torch.arange(-(-n // 4), device=DEV))
    hi, lo = step(hi ^ key[0], lo ^ key[1])
    del key
    share = math.floor((1 - case["p"]) * 65_536 + 0.5)
    out = torch.zeros(n, dtype=torch.float64, device=DEV) if res is None else res.double()
    for j, word in enumerate((lo & 0xFFFF, lo >> 16, hi & 0xFFFF, hi >> 16)):
        part = out[j::4]
        kept = word[:part.numel()] < share
        part += torch.where(kept, x[j::4].double() * (65_536 / max(share, 1)), 0.0)
    return [out]
