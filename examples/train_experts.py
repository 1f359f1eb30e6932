"""A training step of a small recommender with an expert block, on one GPU.

Embedding tables feed a residual block: each sample's concatenated rows x go to
the experts that a router picks, come back weighted, and join the residual
stream through a gated norm; a linear head predicts the click.  Every gradient
is formed by the library's calls and torch's matrix products, the global norm
of all of them (dense parameters and the touched rows of the tables) is clipped
once, and the step follows.

    python examples/train_experts.py [--steps 30] [--batch 4096] [--dim 64]
                                     [--hidden 512] [--dropout 0.1]

The step: prepare and look up (emb_bag_prepare, emb_bag_forward_prepared), route
(emb_expert_sort, _dispatch, _combine), join (emb_gated_norm_forward), their
gradients in reverse, with experts of one matrix each or, given a hidden width, gated
feed-forward blocks (emb_gated_ffn_forward, _backward), dropout of what they
return (emb_dropout), the tables' deduplicated gradients
(emb_bag_grad_reduce_prepared), the clip (emb_clip_grad_norm), and the Adagrad
step of the rows with the clipped sums (emb_bag_adagrad_reduced_prepared).
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from recommender_embedding_tables_amd import embtab as eb  # noqa: E402

GATE = eb.EMB_GATE_ROW | eb.EMB_GATE_SIGMOID
NORM_EPS, ADAGRAD_EPS = 1e-6, 1e-8
PARAMS = ("router", "experts", "gate", "post", "scale", "pre", "head")
FFN_PARAMS = ("router", "w_in", "w_out", "gate", "post", "scale", "pre", "head")


class Model:
    """Parameters, buffers and workspaces, allocated once for a batch size."""

    def __init__(self, rows, dim, batch, experts=8, topk=2, max_norm=1.0, lr=0.05, seed=1,
                 device="cuda", hidden=0, dropout=0.0):
        self.tabs = eb.EmbTables(rows, dim, seed=seed, device=device)
        self.batch, self.experts, self.topk = batch, experts, topk
        self.width = width = self.tabs.T * dim
        self.capacity = -(-batch * topk * 5 // (4 * experts))  # 1.25 times an even share
        self.rows_m = experts * self.capacity
        self.max_norm, self.lr = max_norm, lr
        self.hidden, self.dropout = hidden, dropout
        self.names = FFN_PARAMS if hidden else PARAMS
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def normal(*shape):
            return torch.randn(*shape, generator=g, device=device) / shape[-2] ** 0.5

        ones = torch.ones(width, device=device)
        if hidden:  # rows are outputs, as emb_gated_ffn_forward takes them
            block = {"w_in": normal(experts, width, 2 * hidden).transpose(1, 2).contiguous(),
                     "w_out": normal(experts, hidden, width).transpose(1, 2).contiguous()}
        else:
            block = {"experts": normal(experts, width, width)}
        self.p = {"router": normal(width, experts), **block,
                  "gate": normal(width, 1).view(-1), "post": ones.clone(), "scale": 0.5 * ones,
                  "pre": ones.clone(), "head": normal(width, 1).view(-1)}
        # gradients, clipped in place
        self.g = {k: torch.zeros_like(v) for k, v in self.p.items()}
        self.grads = eb.TensorList([self.g[k] for k in self.names])

        def f(*shape, dtype=torch.float32):
            return torch.empty(shape, dtype=dtype, device=device)

        b, m = batch, self.rows_m
        i32 = dict(dtype=torch.int32)
        self.x, self.block, self.y, self.h = (f(b, width) for _ in range(4))
        self.dx, self.dblock, self.dtok = (f(b, width) for _ in range(3))
        self.xs, self.dys = f(m, width), f(m, width)
        self.dgate, self.dchoice = f(b), f(b, topk)
        self.offsets, self.src, self.pos = f(experts + 1, **i32), f(m, **i32), f(b, topk, **i32)
        self.norm, self.sqnorm = f(2), f(1, dtype=torch.float64)
        need = max(eb.emb_expert_workspace_bytes(b, topk, experts),
                   eb.emb_gated_norm_workspace_bytes(b, width),
                   eb.emb_grad_workspace_bytes(self.grads))
        if hidden:
            self.ys, self.dxs = f(m, width), f(m, width)
            self.gu, self.act = f(m, 2 * hidden), f(m, hidden)
            need = max(need, eb.emb_gated_ffn_workspace_bytes(m, experts, width, hidden,
                                                              eb.EMB_F32))
        self.ws = f(need, dtype=torch.uint8)
        # seed and counter of the dropout's random words, of this step and the next
        self.rng = torch.tensor([seed, 0], device=device)
        self.shape = (b, topk, m, width, eb.EMB_F32)

    def ffn_shape(self):
        return (self.rows_m, self.experts, self.capacity, self.width, self.hidden, eb.EMB_F32,
                eb.EMB_ACT_SILU)

    def drop(self, x):
        """Dropout in place, of the block forward and of its gradient backward."""
        eb.check(eb.emb_dropout(x, None, x.numel(), eb.EMB_F32, self.dropout, self.rng, x),
                 "dropout")

    # ------------------------------------------------------------ forward
    def forward(self, offsets, ids):
        t, p, nnz = self.tabs, self.p, ids.numel()
        self.table_ws, self.table_bytes = t.workspace(self.batch, nnz)
        eb.check(eb.emb_bag_prepare(t.handle, offsets, ids, self.batch, nnz, eb.EMB_POOL_SUM,
                                    self.table_ws, self.table_bytes), "prepare")
        eb.check(eb.emb_bag_forward_prepared(t.handle, offsets, ids, self.batch, nnz,
                                             eb.EMB_POOL_SUM, self.x, self.table_ws,
                                             self.table_bytes), "lookup")
        top, self.choice = torch.topk(self.x @ p["router"], self.topk, dim=1)
        self.weight = torch.softmax(top, 1)
        eb.check(eb.emb_expert_sort(self.choice, self.batch, self.topk, self.experts,
                                    self.capacity, self.offsets, self.src, self.pos, self.ws,
                                    self.ws.numel()), "sort")
        eb.check(eb.emb_expert_dispatch(self.x, self.pos, self.src, *self.shape, self.xs),
                 "dispatch")
        if self.hidden:
            eb.check(eb.emb_gated_ffn_forward(self.xs, p["w_in"], p["w_out"], self.offsets,
                                              *self.ffn_shape(), self.gu, self.act, self.ys,
                                              self.ws, self.ws.numel()), "experts")
        else:
            self.ys = torch.bmm(self.xs.view(self.experts, self.capacity, self.width),
                                p["experts"])
        eb.check(eb.emb_expert_combine(self.ys, self.pos, self.weight, *self.shape, self.block),
                 "combine")
        if self.dropout:
            self.drop(self.block)
        self.a = self.x @ p["gate"]
        eb.check(eb.emb_gated_norm_forward(self.x, self.block, self.a, p["post"], p["scale"],
                                           p["pre"], self.batch, self.width, eb.EMB_F32, GATE,
                                           NORM_EPS, self.y, self.h), "norm")
        return self.h @ p["head"] + self.y.mean(1)

    # ------------------------------------------------------------ backward
    def backward(self, dlogit):
        """Gradients into self.g and, of the lookup's output, returned."""
        p, g, e = self.p, self.g, self.experts
        torch.mv(self.h.t(), dlogit, out=g["head"])
        dh = torch.outer(dlogit, p["head"])
        dy = (dlogit / self.width)[:, None].expand(-1, self.width).contiguous()
        eb.check(eb.emb_gated_norm_backward(
            self.y, self.block, self.a, p["post"], p["scale"], p["pre"], dy, dh, self.batch,
            self.width, eb.EMB_F32, GATE, NORM_EPS, self.dx, self.dblock, self.dgate, g["post"],
            g["scale"], g["pre"], self.ws, self.ws.numel()), "norm backward")
        if self.dropout:  # the forward's random words again
            self.drop(self.dblock)
        eb.check(eb.emb_expert_combine_backward(self.dblock, self.ys, self.pos, self.src,
                                                self.weight, *self.shape, self.dys, self.dchoice),
                 "combine backward")
        if self.hidden:
            dxs = self.dxs
            eb.check(eb.emb_gated_ffn_backward(self.xs, self.gu, self.act, p["w_in"], p["w_out"],
                                               self.dys, self.offsets, *self.ffn_shape(), dxs,
                                               g["w_in"], g["w_out"], self.ws, self.ws.numel()),
                     "experts backward")
        else:
            dys = self.dys.view(e, self.capacity, self.width)
            xs = self.xs.view(e, self.capacity, self.width)
            torch.bmm(xs.transpose(1, 2).contiguous(), dys, out=g["experts"])
            dxs = torch.bmm(dys, p["experts"].transpose(1, 2).contiguous())
        eb.check(eb.emb_expert_dispatch_backward(dxs, self.pos, *self.shape, self.dtok),
                 "dispatch backward")
        # the router: through the softmax over the chosen logits
        w = self.weight
        dtop = w * (self.dchoice - (w * self.dchoice).sum(1, keepdim=True))
        dlogits = torch.zeros(self.batch, e, device=w.device).scatter_(1, self.choice, dtop)
        torch.mm(self.x.t(), dlogits, out=g["router"])
        torch.mv(self.x.t(), self.dgate, out=g["gate"])
        return self.dx + self.dtok + dlogits @ p["router"].t() + torch.outer(self.dgate, p["gate"])

    def step(self, offsets, ids, labels):
        """One training step; returns (loss, norm and coefficient) as device tensors."""
        t, nnz = self.tabs, ids.numel()
        logits = self.forward(offsets, ids)
        loss = F.binary_cross_entropy_with_logits(logits, labels)
        self.dpooled = self.backward((torch.sigmoid(logits) - labels) / self.batch)
        self.sums = torch.empty(min(nnz, t.total_rows), t.D, device=logits.device)
        eb.check(eb.emb_bag_grad_reduce_prepared(t.handle, self.batch, nnz, eb.EMB_POOL_SUM,
                                                 self.dpooled, self.sums, self.sqnorm,
                                                 self.table_ws, self.table_bytes), "reduce")
        eb.check(eb.emb_clip_grad_norm(self.grads, self.grads, self.sqnorm, 1, self.max_norm,
                                       self.norm, self.ws, self.ws.numel()), "clip")
        for k in self.names:
            self.p[k].add_(self.g[k], alpha=-self.lr)
        eb.check(eb.emb_bag_adagrad_reduced_prepared(t.handle, self.batch, nnz, self.sums,
                                                     self.norm[1:], self.lr, ADAGRAD_EPS,
                                                     self.table_ws, self.table_bytes), "step")
        self.rng[1] += (self.block.numel() + 3) // 4  # past this step's random words
        return loss, self.norm

    def close(self):
        self.tabs.close()


def batch_of(rows, batch, seed, device="cuda"):
    """One-hot ids (popular rows more often) and labels that depend on them."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    n = torch.tensor(rows, device=device)[:, None]
    u = torch.rand(len(rows), batch, generator=g, device=device)
    ids = torch.clamp((u ** 3 * n).to(torch.int64), max=n - 1)
    labels = ((ids * 2654435761 >> 7) % 2).sum(0) > len(rows) // 2
    offsets = torch.arange(len(rows) * batch + 1, device=device)
    return offsets, ids.reshape(-1), labels.float()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--batch", type=int, default=4096)
    ap.add_argument("--dim", type=int, default=64)
    ap.add_argument("--rows", type=int, nargs="+", default=[50, 200, 1000, 5000])
    ap.add_argument("--hidden", type=int, default=0, help="of gated feed-forward experts")
    ap.add_argument("--dropout", type=float, default=0.0)
    a = ap.parse_args(argv)
    model = Model(a.rows, a.dim, a.batch, hidden=a.hidden, dropout=a.dropout)
    losses = []
    for i in range(a.steps):
        loss, norm = model.step(*batch_of(a.rows, a.batch, i))
        losses.append(float(loss))
        print(f"step {i:3d}  loss {losses[-1]:.4f}  gradient norm {float(norm[0]):.3f}  "
              f"scaled by {float(norm[1]):.3f}", flush=True)
    status, _ = eb.emb_status_sync(model.tabs.handle)
    eb.check(status, "status")
    model.close()
    return losses


if __name__ == "__main__":
    main()
