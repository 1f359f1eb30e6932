"""What is measured of the training-step operators beside the embedding path.

Three families, each in the directions a training step runs them:

  clip        the global norm of a list of dense gradients, and the list
              scaled by min(1, max_norm / (norm + 1e-6));
  tables      the same norm over the deduplicated gradients of embedding
              tables together with a dense list, then the Adagrad step of the
              touched rows with the clipped gradient;
  route       choices sorted by expert, the rows copied into expert order and
              the experts' rows combined back with their weights;
  route_grad  the gradients of the combine and of the copy;
  norm        a block's output normalised, gated, scaled and added to the
              residual, and the norm of the sum for the next block;
  norm_grad   its gradients.

`run` takes the plain torch form where `own` is false and the library's entry
points where it is true.  `exact` gives the outputs in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
LR, EPS = 0.01, 1e-8
NORM_EPS = 1e-6


def listed():
    return [
        # the biases and small layers of a tower on a short batch: latency
        {"name": "clip_12_small_f32", "op": "clip", "tensors": 12, "elements": 60_000,
         "kind": "f32", "out": "f32", "max_norm": 1.0, "layout": 1},
        # every weight and bias of a large dense part, bf16 and fp32 gradients
        # as a mixed-precision backward leaves them, clipped into fp32
        {"name": "clip_60_mixed", "op": "clip", "tensors": 60, "elements": 256_000_000,
         "kind": "mixed", "out": "f32", "max_norm": 1.0, "layout": 2},
        # multi-hot mean bags at D = 64 with a small tower beside the tables
        {"name": "tables_8x64_bags", "op": "tables", "tables": 8, "dim": 64, "batch": 2048,
         "rows_lo": 50_000, "rows_hi": 50_000, "bag": 20, "mean": True, "tensors": 12,
         "elements": 500_000, "max_norm": 1.0, "layout": 3},
        # 26 one-hot tables at D = 128 and the full batch
        {"name": "tables_26x128_one_hot", "op": "tables", "tables": 26, "dim": 128,
         "batch": 65_536, "rows_lo": 100, "rows_hi": 300_000, "bag": 1, "mean": False,
         "tensors": 24, "elements": 4_000_000, "max_norm": 1.0, "layout": 4},
        # a serving batch: 64 samples, two of eight experts: latency
        {"name": "route_64x512_bf16", "op": "route", "tokens": 64, "topk": 2, "experts": 8,
         "capacity": 0, "dim": 512, "kind": "bf16", "absent": 0.0},
        # the concatenated pooled rows of 26 tables (26 * 128 wide), 64 experts
        {"name": "route_65536x3328_bf16", "op": "route", "tokens": 65_536, "topk": 2,
         "experts": 64, "capacity": 0, "dim": 3328, "kind": "bf16", "absent": 0.02},
        # the interaction's output width (odd), experts at a fixed capacity
        {"name": "route_grad_16384x479_f32", "op": "route_grad", "tokens": 16_384, "topk": 2,
         "experts": 32, "capacity": 1280, "dim": 479, "kind": "f32", "absent": 0.0},
        {"name": "route_grad_16384x3328_bf16", "op": "route_grad", "tokens": 16_384, "topk": 4,
         "experts": 64, "capacity": 0, "dim": 3328, "kind": "bf16", "absent": 0.02},
        # one small batch of the interaction's output, a gate value per row
        {"name": "norm_256x479_f32", "op": "norm", "rows": 256, "dim": 479, "kind": "f32",
         "gate": "row", "sigmoid": True, "post": True},
        # the concatenated pooled rows, an element-wise sigmoid gate
        {"name": "norm_32768x3328_bf16", "op": "norm", "rows": 32_768, "dim": 3328,
         "kind": "bf16", "gate": "element", "sigmoid": True, "post": True},
        {"name": "norm_grad_4096x512_f32", "op": "norm_grad", "rows": 4096, "dim": 512,
         "kind": "f32", "gate": "row", "sigmoid": True, "post": True},
        {"name": "norm_grad_16384x3328_bf16", "op": "norm_grad", "rows": 16_384, "dim": 3328,
         "kind": "bf16", "gate": "element", "sigmoid": True, "post": True},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["clip", "tables", "route", "route_grad", "norm", "norm_grad"])
    if op == "clip":
        n = log(1, 60)
        return {"op": op, "tensors": n, "elements": max(8 * n, log(1000, 128_000_000)),
                "kind": rng.choice(["f32", "bf16", "f16", "mixed"]),
                "out": rng.choice(["f32", "same"]), "max_norm": rng.choice([0.5, 1.0, 1e6]),
                "layout": rng.randrange(1 << 20)}
    if op == "tables":
        t, bag = rng.randint(1, 26), rng.choice([1, 1, 2, 5, 20])
        dim = rng.choice([16, 32, 64, 128, 256])
        most = 65_536 * 26 * 128 // 4  # occurrences times width
        batch = max(3, min(log(50, 65_536), most // (t * bag * dim)))
        lo = log(20, 2000)
        return {"op": op, "tables": t, "dim": dim, "batch": batch, "rows_lo": lo,
                "rows_hi": max(lo, log(1000, 100_000)), "bag": bag, "mean": rng.random() < 0.5,
                "tensors": rng.randint(1, 40), "elements": log(2000, 4_000_000),
                "max_norm": rng.choice([0.5, 1.0, 1e6]), "layout": rng.randrange(1 << 20)}
    if op in ("route", "route_grad"):
        e = rng.choice([2, 4, 8, 16, 32, 64, 100, 256])
        k = rng.randint(1, min(e, 8))
        dim = rng.choice([64, 128, 351, 479, 512, 1000, 1664, 3328, log(33, 4000)])
        most = 65_536 * 2 * 3328 // 4
        n = max(1, min(log(1, 65_536), most // (k * dim)))
        cap = 0 if rng.random() < 0.6 else max(1, int(n * k / e * rng.uniform(0.8, 1.5)))
        return {"op": op, "tokens": n, "topk": k, "experts": e, "capacity": cap, "dim": dim,
                "kind": rng.choice(["f32", "bf16", "f16"]), "absent": rng.choice([0.0, 0.02, 0.3])}
    dim = rng.choice([64, 128, 351, 479, 512, 1000, 1664, 3328, log(17, 8000)])
    most = 16_384 * 3328 // 2
    return {"op": op, "rows": max(1, min(log(1, 65_536), most // dim)), "dim": dim,
            "kind": rng.choice(["f32", "bf16", "f16"]),
            "gate": rng.choice(["none", "row", "element"]), "sigmoid": rng.random() < 0.5,
            "post": rng.random() < 0.7}


# ---------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _sizes(case):
    """Sizes of the dense list: weights of spread sizes, a short odd bias after each."""
    n, total, r = case["tensors"], case["elements"], random.Random(case["layout"])
    w = [r.uniform(0.2, 4.0) if i % 2 == 0 else 0.0 for i in range(n)]
    s = sum(w)
    return [max(1, int(total * v / s)) if v else (int(math.sqrt(total / n)) | 1) for v in w]


def _dense(case, g):
    """Gradients: normal values, each tensor at a scale of its own."""
    kind = case.get("kind", "f32")
    sizes = _sizes(case)
    scale = torch.exp(torch.rand(len(sizes), generator=g, device=DEV) * 4 - 6)
    flat = torch.randn(sum(sizes), generator=g, device=DEV)
    names = [kind if kind != "mixed" else ("bf16" if i % 3 else "f32") for i in range(len(sizes))]
    return [(x * scale[i]).to(DTYPES[names[i]])
            for i, x in enumerate(torch.split(flat, sizes))]


def _table_rows(case):
    t, lo, hi = case["tables"], case["rows_lo"], case["rows_hi"]
    return [int(round(lo * (hi / lo) ** (i / max(1, t - 1)))) for i in range(t)]


def _table_inputs(case, g):
    rows = _table_rows(case)
    t, b, d = case["tables"], case["batch"], case["dim"]
    if case["bag"] == 1:
        lens = torch.ones(t * b, dtype=torch.int64, device=DEV)
    else:  # 1 .. 2 * bag - 1 ids, an empty bag now and then
        lens = torch.randint(0, 2 * case["bag"], (t * b,), generator=g, device=DEV)
    offsets = torch.zeros(t * b + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = torch.cumsum(lens, 0)
    nnz = int(offsets[-1])
    bag = torch.repeat_interleave(torch.arange(t * b, device=DEV), lens, output_size=nnz)
    n = torch.tensor(rows, device=DEV)
    # popular ids: the cube of a uniform number
    u = torch.rand(nnz, generator=g, device=DEV, dtype=torch.float64)
    ids = torch.clamp((u ** 3 * n[bag // b]).to(torch.int64), max=n[bag // b] - 1)
    weights = torch.randn(sum(rows), d, generator=g, device=DEV) * 0.05
    accum = torch.rand(sum(rows), d, generator=g, device=DEV) * 0.1 + 0.1
    grad = torch.randn(b, t, d, generator=g, device=DEV) * 0.01
    return rows, offsets, ids, lens, bag, weights, accum, grad


def _route_inputs(case, g):
    n, k, e, d = case["tokens"], case["topk"], case["experts"], case["dim"]
    t = DTYPES[case["kind"]]
    m = n * k if not case["capacity"] else e * case["capacity"]
    # some experts are liked better than others
    logits = torch.randn(n, e, generator=g, device=DEV) + torch.randn(e, generator=g, device=DEV)
    top, ids = torch.topk(logits, k, dim=1)
    weights = torch.softmax(top, 1)
    gone = torch.rand(n, 1, generator=g, device=DEV) < case["absent"]  # padded samples
    ids = torch.where(gone, -2, ids).contiguous()
    rows = [torch.randn(s, d, generator=g, device=DEV).to(t) for s in (n, m, m)]
    return ids, weights, rows, m


def _norm_inputs(case, g):
    n, d, t = case["rows"], case["dim"], DTYPES[case["kind"]]
    x = torch.randn(n, d, generator=g, device=DEV)
    block = torch.randn(n, d, generator=g, device=DEV) * 3
    gate = {"none": None, "row": torch.randn(n, generator=g, device=DEV),
            "element": torch.randn(n, d, generator=g, device=DEV)}[case["gate"]]
    w_post, scale, w_pre = (1 + 0.1 * torch.randn(3, d, generator=g, device=DEV)).unbind(0)
    dy = torch.randn(n, d, generator=g, device=DEV)
    dh = torch.randn(n, d, generator=g, device=DEV)
    cast = [None if v is None else v.to(t) for v in (x, block, gate, dy, dh)]
    return cast, (w_post.contiguous() if case["post"] else None), (0.5 * scale).contiguous(), \
        w_pre.contiguous()


# ---------------------------------------------------------------- prepare

def prepare(case, seed):
    g = _generator(seed)
    s = {"case": case}
    if case["op"] == "clip":
        s["grads"] = _dense(case, g)
        s["out"] = [torch.empty_like(x, dtype=torch.float32 if case["out"] == "f32" else x.dtype)
                    for x in s["grads"]]
    elif case["op"] == "tables":
        rows, offsets, ids, lens, bag, weights, accum, grad = _table_inputs(case, g)
        s.update(rows=rows, offsets=offsets, ids=ids, lens=lens, bag=bag, grad=grad,
                 grads=_dense(case, g))
        s["out"] = [torch.empty_like(x) for x in s["grads"]]
        s["starts"] = torch.tensor([sum(rows[:i]) for i in range(len(rows))], device=DEV)
        s["weights"], s["accum"] = weights, accum
    elif case["op"] in ("route", "route_grad"):
        ids, w, (x, a, b), m = _route_inputs(case, g)
        s.update(ids=ids, w=w, x=x, a=a, b=b, m=m)
        if case["op"] == "route_grad":  # the forward's sort, kept for its backward
            s["offsets"], s["src"], s["pos"] = _sorted(ids, case["experts"], case["capacity"], m)
    else:
        (s["x"], s["block"], s["gate"], s["dy"], s["dh"]), s["w_post"], s["scale"], s["w_pre"] = \
            _norm_inputs(case, g)
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """The handle, argument lists, workspaces and output buffers a program keeps."""
    from recommender_embedding_tables_amd import embtab as eb
    case = s["case"]
    i32 = dict(dtype=torch.int32, device=DEV)
    if case["op"] in ("clip", "tables"):
        s["in_list"], s["out_list"] = eb.TensorList(s["grads"]), eb.TensorList(s["out"])
        s["norm"] = torch.empty(2, device=DEV)
        s["ws_bytes"] = eb.emb_grad_workspace_bytes(s["in_list"])
        s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device=DEV)
    if case["op"] == "tables":
        tabs = eb.EmbTables(s["rows"], case["dim"])
        tabs.weights.copy_(s["weights"])
        tabs.accum.copy_(s["accum"])
        s["weights"], s["accum"] = tabs.weights, tabs.accum
        s["tabs"], s["sq"] = tabs, torch.empty(1, dtype=torch.float64, device=DEV)
        s["sums"] = torch.empty(min(s["ids"].numel(), tabs.total_rows), case["dim"], device=DEV)
        s["table_ws"], s["table_ws_bytes"] = tabs.workspace(case["batch"], s["ids"].numel())
    elif case["op"] == "route":
        e = case["experts"]
        s["offsets"] = torch.empty(e + 1, **i32)
        s["src"], s["pos"] = torch.empty(s["m"], **i32), torch.empty(s["ids"].shape, **i32)
        s["xs"], s["y"] = torch.empty_like(s["a"]), torch.empty_like(s["x"])
        s["ws_bytes"] = eb.emb_expert_workspace_bytes(case["tokens"], case["topk"], e)
        s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device=DEV)
    elif case["op"] == "route_grad":
        s["dys"], s["dw"], s["dx"] = (torch.empty_like(s[v]) for v in ("a", "w", "x"))
    elif case["op"] == "norm":
        s["y"], s["h"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
    elif case["op"] == "norm_grad":
        s["dx"], s["dblock"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
        s["dgate"] = None if s["gate"] is None else torch.empty_like(s["gate"])
        s["dparams"] = torch.empty(3, case["dim"], device=DEV)
        s["ws_bytes"] = eb.emb_gated_norm_workspace_bytes(case["rows"], case["dim"])
        s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device=DEV)


# ---------------------------------------------------------------- run

def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _coef(norm, max_norm):
    c = torch.clamp(max_norm / (norm + 1e-6), max=1.0)
    return torch.where(torch.isfinite(norm), c, 0.0).float()


def _square_sum(tensors):
    return torch.stack([x.float().square().sum(dtype=torch.float64) for x in tensors]).sum()


def _scaled(tensors, out, coef):
    return [torch.where(coef == 0, 0.0, x.float() * coef).to(o.dtype)
            for x, o in zip(tensors, out)]


def _clip(s):
    norm = torch.sqrt(_square_sum(s["grads"]))
    coef = _coef(norm, s["case"]["max_norm"])
    return [norm.float(), coef, _scaled(s["grads"], s["out"], coef)]


def _tables(s):
    case = s["case"]
    t, b, d = case["tables"], case["batch"], case["dim"]
    row = s["starts"][s["bag"] // b] + s["ids"]
    uniq, inverse = torch.unique(row, return_inverse=True)
    per_bag = s["grad"].transpose(0, 1).reshape(t * b, d)
    if case["mean"]:
        per_bag = per_bag / torch.clamp(s["lens"], min=1)[:, None]
    g = torch.zeros(uniq.numel(), d, device=DEV).index_add_(0, inverse, per_bag[s["bag"]])
    norm = torch.sqrt(_square_sum(s["grads"] + [g]))
    coef = _coef(norm, case["max_norm"])
    g = torch.where(coef == 0, 0.0, g * coef)
    acc = s["accum"][uniq] + g * g
    s["weights"][uniq] -= LR * g / (torch.sqrt(acc) + EPS)
    s["accum"][uniq] = acc
    return [norm.float(), coef, _scaled(s["grads"], s["out"], coef), s["weights"], s["accum"]]


def _sorted(ids, experts, capacity, m):
    """(offsets, src, pos): kept choices per expert (exclusive sums), the choice
    in each row (-1: none) and the row of each choice (-1: dropped)."""
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    order = torch.argsort(key, stable=True)
    key = key[order]
    count = torch.bincount(key, minlength=experts + 1)
    start = torch.cumsum(count, 0) - count
    rank = torch.arange(flat.numel(), device=DEV) - start[key]
    kept, row = key < experts, start[key] + rank
    if capacity:
        kept, row = kept & (rank < capacity), key * capacity + rank
        count = torch.clamp(count, max=capacity)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.cumsum(count[:experts], 0)
    src = torch.full((m + 1,), -1, dtype=torch.int32, device=DEV)
    src[torch.where(kept, row, m)] = torch.where(kept, order, -1).int()
    pos = torch.empty(flat.numel(), dtype=torch.int32, device=DEV)
    pos[order] = torch.where(kept, row, -1).int()
    return offsets, src[:m], pos.reshape(ids.shape)


def _rows_of(values, pos):
    """values[pos] in 32 bits, zero where pos is -1."""
    got = values[torch.clamp(pos, min=0).long()].float()
    return torch.where((pos >= 0)[..., None], got, 0.0)


def _route(s):
    case = s["case"]
    offsets, src, pos = _sorted(s["ids"], case["experts"], case["capacity"], s["m"])
    token = torch.where(src >= 0, src // case["topk"], -1)
    xs = _rows_of(s["x"], token).to(s["x"].dtype)
    y = (s["w"][..., None] * _rows_of(s["a"], pos)).sum(1).to(s["x"].dtype)
    return [offsets, src, pos, xs, y]


def _route_grad(s):
    k, t = s["case"]["topk"], s["x"].dtype
    dy, ys, dxs, src, pos = s["x"], s["a"], s["b"], s["src"], s["pos"]
    token = torch.where(src >= 0, src // k, -1)
    w = s["w"].reshape(-1)[torch.clamp(src, min=0).long()]
    dys = (w[:, None] * _rows_of(dy, token)).to(t)
    dw = (dy.float()[:, None, :] * _rows_of(ys, pos)).sum(2)
    dx = _rows_of(dxs, pos).sum(1).to(t)
    return [dys, dw, dx]


def _norm_parts(s):
    o = s["block"].float()
    r = torch.rsqrt((o * o).mean(1, keepdim=True) + NORM_EPS) if s["w_post"] is not None else None
    hat = o if r is None else o * r
    u = hat if r is None else hat * s["w_post"]
    a = None if s["gate"] is None else s["gate"].float()
    if a is not None and s["case"]["sigmoid"]:
        a = 1 / (1 + torch.exp(-a))
    if a is not None and a.dim() == 1:
        a = a[:, None]
    return r, hat, u, a


def _norm(s):
    _, _, u, a = _norm_parts(s)
    y = s["x"].float() + (s["scale"] * u if a is None else s["scale"] * a * u)
    r = torch.rsqrt((y * y).mean(1, keepdim=True) + NORM_EPS)
    t = s["x"].dtype
    return [y.to(t), (y * r * s["w_pre"]).to(t)]


def _norm_grad(s):
    t, d = s["x"].dtype, s["case"]["dim"]
    r, hat, u, a = _norm_parts(s)
    y, dy, dh = s["x"].float(), s["dy"].float(), s["dh"].float()  # x stands for the sum y
    ry = torch.rsqrt((y * y).mean(1, keepdim=True) + NORM_EPS)
    yhat, q = y * ry, dh * s["w_pre"]
    dy = dy + ry * (q - yhat * ((q * yhat).sum(1, keepdim=True) / d))
    da = dy * s["scale"] * u
    ga = dy if a is None else dy * a
    du = s["scale"] * ga
    do = du
    if r is not None:
        q = du * s["w_post"]
        do = r * (q - hat * ((q * hat).sum(1, keepdim=True) / d))
    dgate = None
    if a is not None:
        if s["gate"].dim() == 1:
            da = da.sum(1, keepdim=True)
        dgate = (da * a * (1 - a) if s["case"]["sigmoid"] else da).reshape(s["gate"].shape).to(t)
    sums = [None if r is None else (du * hat).sum(0), (ga * u).sum(0), (dh * yhat).sum(0)]
    return [v for v in [dy.to(t), do.to(t), dgate] + sums if v is not None]


_plain = {"clip": _clip, "tables": _tables, "route": _route, "route_grad": _route_grad,
          "norm": _norm, "norm_grad": _norm_grad}


def _own_clip(s):
    from recommender_embedding_tables_amd import embtab as eb
    eb.check(eb.emb_clip_grad_norm(s["in_list"], s["out_list"], None, 0, s["case"]["max_norm"],
                                   s["norm"], s["ws"], s["ws_bytes"]), "clip_grad_norm")
    return [s["norm"][0], s["norm"][1], s["out"]]


def _own_tables(s):
    from recommender_embedding_tables_amd import embtab as eb
    case, h = s["case"], s["tabs"].handle
    b, nnz, ws, n = case["batch"], s["ids"].numel(), s["table_ws"], s["table_ws_bytes"]
    pool = eb.EMB_POOL_MEAN if case["mean"] else eb.EMB_POOL_SUM
    eb.check(eb.emb_bag_prepare(h, s["offsets"], s["ids"], b, nnz, pool, ws, n), "prepare")
    eb.check(eb.emb_bag_grad_reduce_prepared(h, b, nnz, pool, s["grad"], s["sums"], s["sq"], ws, n),
             "grad_reduce")
    eb.check(eb.emb_clip_grad_norm(s["in_list"], s["out_list"], s["sq"], 1, case["max_norm"],
                                   s["norm"], s["ws"], s["ws_bytes"]), "clip_grad_norm")
    eb.check(eb.emb_bag_adagrad_reduced_prepared(h, b, nnz, s["sums"], s["norm"][1:], LR, EPS, ws,
                                                 n), "adagrad_reduced")
    return [s["norm"][0], s["norm"][1], s["out"], s["weights"], s["accum"]]


def _own_route(s):
    from recommender_embedding_tables_amd import embtab as eb
    c = s["case"]
    n, k, e, d = c["tokens"], c["topk"], c["experts"], c["dim"]
    t = eb.dtype_code(s["x"].dtype)
    eb.check(eb.emb_expert_sort(s["ids"], n, k, e, c["capacity"], s["offsets"], s["src"], s["pos"],
                                s["ws"], s["ws_bytes"]), "expert_sort")
    eb.check(eb.emb_expert_dispatch(s["x"], s["pos"], s["src"], n, k, s["m"], d, t, s["xs"]),
             "expert_dispatch")
    eb.check(eb.emb_expert_combine(s["a"], s["pos"], s["w"], n, k, s["m"], d, t, s["y"]),
             "expert_combine")
    return [s["offsets"], s["src"], s["pos"], s["xs"], s["y"]]


def _own_route_grad(s):
    from recommender_embedding_tables_amd import embtab as eb
    c = s["case"]
    n, k, d = c["tokens"], c["topk"], c["dim"]
    t = eb.dtype_code(s["x"].dtype)
    eb.check(eb.emb_expert_combine_backward(s["x"], s["a"], s["pos"], s["src"], s["w"], n, k,
                                            s["m"], d, t, s["dys"], s["dw"]), "combine_backward")
    eb.check(eb.emb_expert_dispatch_backward(s["b"], s["pos"], n, k, s["m"], d, t, s["dx"]),
             "dispatch_backward")
    return [s["dys"], s["dw"], s["dx"]]


def _gate_kind(s, eb):
    if s["gate"] is None:
        return eb.EMB_GATE_NONE
    kind = eb.EMB_GATE_ROW if s["gate"].dim() == 1 else eb.EMB_GATE_ELEMENT
    return kind | (eb.EMB_GATE_SIGMOID if s["case"]["sigmoid"] else 0)


def _own_norm(s):
    from recommender_embedding_tables_amd import embtab as eb
    c = s["case"]
    eb.check(eb.emb_gated_norm_forward(
        s["x"], s["block"], s["gate"], s["w_post"], s["scale"], s["w_pre"], c["rows"], c["dim"],
        eb.dtype_code(s["x"].dtype), _gate_kind(s, eb), NORM_EPS, s["y"], s["h"]), "gated_norm")
    return [s["y"], s["h"]]


def _own_norm_grad(s):
    from recommender_embedding_tables_amd import embtab as eb
    c, (dw_post, dscale, dw_pre) = s["case"], s["dparams"]
    dw_post = dw_post if c["post"] else None
    eb.check(eb.emb_gated_norm_backward(
        s["x"], s["block"], s["gate"], s["w_post"], s["scale"], s["w_pre"], s["dy"], s["dh"],
        c["rows"], c["dim"], eb.dtype_code(s["x"].dtype), _gate_kind(s, eb), NORM_EPS, s["dx"],
        s["dblock"], s["dgate"], dw_post, dscale, dw_pre, s["ws"], s["ws_bytes"]),
        "gated_norm_backward")
    return [v for v in (s["dx"], s["dblock"], s["dgate"], dw_post, dscale, dw_pre)
            if v is not None]


_own = {"clip": _own_clip, "tables": _own_tables, "route": _own_route,
        "route_grad": _own_route_grad, "norm": _own_norm, "norm_grad": _own_norm_grad}


# ---------------------------------------------------------------- work

def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2, "mixed": 8 / 3}
    if case["op"] in ("clip", "tables"):
        n = sum(_sizes(case))
        i = size[case.get("kind", "f32")]
        dense = n * (i + (4 if case.get("out", "f32") == "f32" else i))
        if case["op"] == "clip":
            return {"bytes": int(dense), "flops": 3 * n}
        bags = case["tables"] * case["batch"]
        nnz = bags if case["bag"] == 1 else int(bags * (case["bag"] - 0.5))
        # distinct rows of nnz draws of cubed uniform numbers over r rows, by their expectation
        rows, per = _table_rows(case), nnz / case["tables"]
        touched = 0.0
        for r in rows:
            edges = [(j / 256) ** (1 / 3) for j in range(257)]
            touched += sum(r / 256 * -math.expm1(-per * (b - a) * 256 / r)
                           for a, b in zip(edges, edges[1:]))
        d = case["dim"]
        return {"bytes": int(dense + 8 * (nnz + bags) + 4 * d * bags + 16 * d * touched),
                "flops": int(3 * n + d * (2 * nnz + 12 * touched))}
    if case["op"] in ("route", "route_grad"):
        n, k, d, i = case["tokens"], case["topk"], case["dim"], size[case["kind"]]
        kept = n * k * (1 - case["absent"])
        m = n * k if not case["capacity"] else case["experts"] * case["capacity"]
        if case["capacity"]:
            kept = min(kept, m)
        if case["op"] == "route":  # x and the kept rows read, xs and y written
            b = i * d * (2 * n + kept + m) + 12 * n * k + 4 * m + 4 * n * k
            return {"bytes": int(b), "flops": int(2 * kept * d)}
        b = i * d * (2 * n + 2 * kept + m) + 16 * n * k + 4 * m
        return {"bytes": int(b), "flops": int(4 * kept * d)}
    n, d, i = case["rows"], case["dim"], size[case["kind"]]
    e = {"none": 0, "row": 0, "element": 1}[case["gate"]]
    streams = 4 + e if case["op"] == "norm" else 6 + 2 * e
    return {"bytes": i * n * d * streams + 12 * d, "flops": (12 if case["op"] == "norm" else 30) * n * d}


# ---------------------------------------------------------------- exact

def exact(case, seed):
    g = _generator(seed)
    return {"clip": _exact_clip, "tables": _exact_tables, "route": _exact_route,
            "route_grad": _exact_route, "norm": _exact_norm, "norm_grad": _exact_norm}[
                case["op"]](case, g)


def _exact_scale(total, max_norm):
    norm = total ** 0.5
    return norm, min(1.0, max_norm / (norm + 1e-6))


def _exact_clip(case, g):
    grads = [x.double() for x in _dense(case, g)]
    norm, coef = _exact_scale(sum(float(x.dot(x)) for x in grads), case["max_norm"])
    one = torch.tensor([norm, coef], dtype=torch.float64, device=DEV)
    return [one[0], one[1], [x * coef for x in grads]]


def _exact_tables(case, g):
    rows, offsets, ids, lens, bag, weights, accum, grad = _table_inputs(case, g)
    dense = [x.double() for x in _dense(case, g)]
    w, acc = weights.double(), accum.double()
    b, d = case["batch"], case["dim"]
    full = torch.zeros_like(w)
    touched = torch.zeros(w.shape[0], dtype=torch.bool, device=DEV)
    base = 0
    for t, r in enumerate(rows):  # one table after another
        o = offsets[t * b:(t + 1) * b + 1]
        mine = ids[o[0]:o[-1]] + base
        sample = bag[o[0]:o[-1]] - t * b
        per = grad[:, t, :].double()
        if case["mean"]:
            per = per / torch.clamp(o[1:] - o[:-1], min=1).double()[:, None]
        full.index_add_(0, mine, per[sample])
        touched[mine] = True
        base += r
    total = sum(float(x.dot(x)) for x in dense) + float((full * full).sum())
    norm, coef = _exact_scale(total, case["max_norm"])
    full *= coef
    acc = torch.where(touched[:, None], acc + full * full, acc)
    w = torch.where(touched[:, None], w - LR * full / (acc.sqrt() + EPS), w)
    one = torch.tensor([norm, coef], dtype=torch.float64, device=DEV)
    return [one[0], one[1], [x * coef for x in dense], w, acc]


def _exact_route(case, g):
    ids, w, (x, a, b), m = _route_inputs(case, g)
    n, k, e, c = case["tokens"], case["topk"], case["experts"], case["capacity"]
    flat = ids.reshape(-1)
    src = torch.full((m,), -1, dtype=torch.int64, device=DEV)
    pos = torch.full((n * k,), -1, dtype=torch.int64, device=DEV)
    kept, at = [0], 0
    for j in range(e):  # one expert after another
        mine = torch.nonzero(flat == j).reshape(-1)
        mine = mine[:c] if c else mine
        first = j * c if c else at
        place = first + torch.arange(mine.numel(), device=DEV)
        src[place], pos[mine] = mine, place
        at += mine.numel()
        kept.append(at)
    pos2 = pos.reshape(n, k)
    have = src >= 0
    out = torch.zeros(m, case["dim"], dtype=torch.float64, device=DEV)
    x = x.double()
    if case["op"] == "route":
        out[have] = x[src[have] // k]
        y = torch.zeros_like(x)
        for j in range(k):
            on = pos2[:, j] >= 0
            y[on] += w[on, j].double()[:, None] * a[pos2[on, j]].double()
        offsets = torch.tensor(kept, dtype=torch.int32, device=DEV)
        return [offsets, src.int(), pos2.int(), out, y]
    out[have] = w.reshape(-1)[src[have]].double()[:, None] * x[src[have] // k]
    dw = torch.zeros(n, k, dtype=torch.float64, device=DEV)
    dx = torch.zeros_like(x)
    for j in range(k):
        on = pos2[:, j] >= 0
        dw[on, j] = (x[on] * a[pos2[on, j]].double()).sum(1)
        dx[on] += b[pos2[on, j]].double()
    return [out, dw, dx]


def _exact_norm(case, g):
    """The definition in float64; its gradients by automatic differentiation."""
    (x, block, gate, dy, dh), w_post, scale, w_pre = _norm_inputs(case, g)
    grad = case["op"] == "norm_grad"
    x, block, gate, w_post, scale, w_pre = (
        None if v is None else v.double().requires_grad_(grad)
        for v in (x, block, gate, w_post, scale, w_pre))

    def rms(v):
        return v / torch.sqrt(v.pow(2).mean(1, keepdim=True) + NORM_EPS)

    u = block if w_post is None else rms(block) * w_post
    if gate is not None:
        a = torch.sigmoid(gate) if case["sigmoid"] else gate
        u = u * (a[:, None] if gate.dim() == 1 else a)
    branch = scale * u
    if not grad:
        y = x + branch
        return [y, rms(y) * w_pre]
    # x holds the sum y here: the norm's gradient reaches it, and through it the branch
    h = rms(x) * w_pre
    dx, dw_pre = torch.autograd.grad(h, (x, w_pre), dh.double())
    dx = dx + dy.double()
    wanted = [v for v in (block, gate, w_post, scale) if v is not None]
    got = dict(zip(map(id, wanted), torch.autograd.grad(branch, wanted, dx)))
    return [v for v in [dx, got[id(block)], got.get(id(gate)), got.get(id(w_post)),
                        got[id(scale)], dw_pre] if v is not None]
