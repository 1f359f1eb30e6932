"""The expert block's operators as they are used together: one step of the example
with gated feed-forward experts and dropout, and a block whose rows travel to the
experts in 8 bits, against automatic differentiation in 64 bits."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
import train_experts as ex  # noqa: E402
from recommender_embedding_tables_amd import embtab as eb  # noqa: E402
from tests.test_gpu_dense import DEV, TYPES, U, gen, half, rand  # noqa: E402
from tests.test_gpu_expert_block import kept  # noqa: E402

ROWS, DIM, BATCH = [3, 20, 300, 70], 16, 256


def rms(v, eps):
    return v / torch.sqrt((v * v).mean(1, keepdim=True) + eps)


def experts64(x, w_in, w_out, choice, pos, weight):
    """Combined outputs of each token's experts; a choice without a row counts for nothing."""
    f = w_out.shape[2]
    out = torch.zeros_like(x)
    for j in range(choice.shape[1]):
        on = torch.nonzero(pos[:, j] >= 0)[:, 0]
        e = choice[on, j]
        pre = torch.matmul(w_in[e], x[on][:, :, None])[:, :, 0]
        a = pre[:, :f] * torch.sigmoid(pre[:, :f]) * pre[:, f:]
        y = torch.matmul(w_out[e], a[:, :, None])[:, :, 0]
        out = out.index_add(0, on, weight[on, j][:, None] * y)
    return out


@pytest.mark.parametrize("hidden,dropout", [(40, 0.25), (96, 0.0), (0, 0.5)])
def test_one_step_of_the_example(hidden, dropout):
    m = ex.Model(ROWS, DIM, BATCH, max_norm=0.05, hidden=hidden, dropout=dropout)
    offsets, ids, labels = ex.batch_of(ROWS, BATCH, 5)
    m.step(offsets, ids, labels)  # the counter has moved on
    rng = m.rng.tolist()
    assert rng[1] == BATCH * m.width // 4
    p0 = {k: v.double().cpu().requires_grad_() for k, v in m.p.items()}
    w0 = m.tabs.weights.double().cpu().requires_grad_()
    loss, norm = m.step(offsets, ids, labels)
    torch.cuda.synchronize()
    starts = torch.tensor([sum(ROWS[:t]) for t in range(len(ROWS))])[:, None]
    x = w0[ids.cpu().view(len(ROWS), BATCH) + starts].transpose(0, 1).reshape(BATCH, -1)
    choice, pos = m.choice.cpu(), m.pos.cpu()
    w = torch.softmax((x @ p0["router"]).gather(1, choice), 1)
    if hidden:
        block = experts64(x, p0["w_in"], p0["w_out"], choice, pos, w)
    else:
        block = torch.zeros_like(x)
        for j in range(m.topk):
            on = torch.nonzero(pos[:, j] >= 0)[:, 0]
            rows = torch.matmul(x[on][:, None, :], p0["experts"][choice[on, j]])[:, 0]
            block = block.index_add(0, on, w[on, j][:, None] * rows)
    if dropout:
        mask, keep = kept(rng, block.numel(), dropout)
        block = block * mask.cpu().view(block.shape) * (65536 / keep)
    a = torch.sigmoid(x @ p0["gate"])[:, None]
    y = x + p0["scale"] * a * (rms(block, ex.NORM_EPS) * p0["post"])
    logits = (rms(y, ex.NORM_EPS) * p0["pre"]) @ p0["head"] + y.mean(1)
    want = torch.nn.functional.binary_cross_entropy_with_logits(logits, labels.double().cpu())
    grads = torch.autograd.grad(want, list(p0.values()) + [w0])

    def close(got, ref, what):
        # normwise: ten stages of sums of at most 256 terms, each within 256 U
        err = float((got.detach().double().cpu() - ref).norm())
        assert err <= 10 * 256 * U * float(ref.norm()), f"{what}: {err / float(ref.norm()):.2e}"

    close(loss.view(1), want.detach().view(1), "loss")
    total = float(sum((g * g).sum() for g in grads)) ** 0.5
    coef = min(1.0, 0.05 / (total + 1e-6))
    close(norm, torch.tensor([total, coef], dtype=torch.float64), "norm")
    for k, g in zip(p0, grads):
        close(m.g[k], coef * g, "gradient of " + k)
        close(m.p[k], (p0[k] - m.lr * coef * g).detach(), k)
    m.close()


def test_main_with_feed_forward_experts(capsys):
    losses = ex.main(["--steps", "3", "--batch", "512", "--dim", "16", "--hidden", "48",
                      "--dropout", "0.1"])
    assert len(losses) == 3 and all(x == x for x in losses)
    assert capsys.readouterr().out.count("gradient norm") == 3


class Block:
    """x + block, normalised to 8 bits, sent to its experts, combined, dropped out and
    added to the residual; and the gradients, the rounding to 8 bits passed over."""

    def __init__(self, n, d, f, e, k, capacity, t, p):
        g = gen(n + d)

        def values(*shape, s=1.0):
            return rand(g, *shape, scale=s).to(t)

        self.n, self.d, self.f, self.e, self.k, self.cap, self.p = n, d, f, e, k, capacity, p
        self.t, self.code = t, eb.dtype_code(t)
        self.x, self.block, self.dout = values(n, d), values(n, d, s=0.5), values(n, d)
        self.w_in, self.w_out = values(e, 2 * f, d, s=d ** -0.5), values(e, d, f, s=f ** -0.5)
        self.norm_w, self.ones = 1 + 0.1 * rand(g, d), torch.ones(d, device=DEV)
        self.choice = torch.topk(rand(g, n, e), k, dim=1).indices
        self.choice[::9] = eb.EMB_ID_ABSENT
        self.weight = torch.softmax(rand(g, n, k), 1)
        self.m = m = capacity * e if capacity else n * k
        self.rng = torch.tensor([11, 300], device=DEV)

        def e_(*shape, dtype=t):
            return torch.full(shape, 77, dtype=dtype, device=DEV)

        i32 = dict(dtype=torch.int32)
        self.offsets, self.src, self.pos = e_(e + 1, **i32), e_(m, **i32), e_(n, k, **i32)
        self.y, self.z, self.out, self.dz, self.dx, self.dh, self.db = (e_(n, d)
                                                                        for _ in range(7))
        self.codes, self.scales = e_(n, d, dtype=torch.int8), e_(n, dtype=torch.float32)
        self.xs, self.ys, self.dys, self.dxs = (e_(m, d) for _ in range(4))
        self.gu, self.a = e_(m, 2 * f), e_(m, f)
        self.dw, self.dparams = e_(n, k, dtype=torch.float32), e_(2, d, dtype=torch.float32)
        self.dw_in, self.dw_out = e_(e, 2 * f, d), e_(e, d, f)
        self.ws = e_(max(eb.emb_expert_workspace_bytes(n, k, e),
                         eb.emb_gated_norm_workspace_bytes(n, d),
                         eb.emb_gated_ffn_workspace_bytes(m, e, d, f, self.code)),
                     dtype=torch.uint8)

    def run(self, stream=None):
        n, d, k, m, c = self.n, self.d, self.k, self.m, self.code
        ws, nb, s = self.ws, self.ws.numel(), dict(stream=stream)
        ffn = (m, self.e, self.cap, d, self.f, c, eb.EMB_ACT_SILU)
        for st in (
                eb.emb_add_norm_int8(self.x, self.block, self.norm_w, n, d, c, 1e-6, self.y,
                                     self.codes, self.scales, **s),
                eb.emb_expert_sort(self.choice, n, k, self.e, self.cap, self.offsets, self.src,
                                   self.pos, ws, nb, **s),
                eb.emb_expert_dispatch_int8(self.codes, self.scales, self.pos, self.src, n, k, m,
                                            d, c, self.xs, **s),
                eb.emb_gated_ffn_forward(self.xs, self.w_in, self.w_out, self.offsets, *ffn,
                                         self.gu, self.a, self.ys, ws, nb, **s),
                eb.emb_expert_combine(self.ys, self.pos, self.weight, n, k, m, d, c, self.z, **s),
                eb.emb_dropout(self.z, self.y, n * d, c, self.p, self.rng, self.out, **s),
                eb.emb_dropout(self.dout, None, n * d, c, self.p, self.rng, self.dz, **s),
                eb.emb_expert_combine_backward(self.dz, self.ys, self.pos, self.src, self.weight,
                                               n, k, m, d, c, self.dys, self.dw, **s),
                eb.emb_gated_ffn_backward(self.xs, self.gu, self.a, self.w_in, self.w_out,
                                          self.dys, self.offsets, *ffn, self.dxs, self.dw_in,
                                          self.dw_out, ws, nb, **s),
                eb.emb_expert_dispatch_backward(self.dxs, self.pos, n, k, m, d, c, self.dh, **s),
                eb.emb_gated_norm_backward(self.y, self.block, None, None, self.ones, self.norm_w,
                                           self.dout, self.dh, n, d, c, eb.EMB_GATE_NONE, 1e-6,
                                           self.dx, self.db, None, None, self.dparams[0],
                                           self.dparams[1], ws, nb, **s)):
            eb.check(st, "block")

    def outputs(self):
        return dict(y=self.y, codes=self.codes, out=self.out, dx=self.dx, dw=self.dw,
                    dw_in=self.dw_in, dw_out=self.dw_out, dnorm=self.dparams[1])


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("n,d,f,e,k,cap", [(300, 72, 100, 6, 2, 0), (200, 479, 96, 4, 2, 120),
                                           (24, 64, 128, 8, 3, 0), (1500, 256, 264, 5, 2, 0)])
def test_block_with_rows_in_8_bits(n, d, f, e, k, cap, kind):
    b = Block(n, d, f, e, k, cap, TYPES[kind], 0.2)
    b.run()
    torch.cuda.synchronize()
    leaf = {name: getattr(b, name).double().cpu().requires_grad_()
            for name in ("x", "block", "w_in", "w_out", "norm_w", "weight")}
    y = leaf["x"] + leaf["block"]
    h = rms(y, 1e-6) * leaf["norm_w"]
    sent = b.codes.double().cpu() * b.scales.double().cpu()[:, None]
    # half a code of the row's largest, and the code's own error below a hundredth of one
    assert ((sent - h).abs() <= 0.51 * h.abs().amax(1, keepdim=True) / 127).all()
    h = h + (sent - h).detach()
    z = experts64(h, leaf["w_in"], leaf["w_out"], b.choice.cpu().clamp(min=0), b.pos.cpu(),
                  leaf["weight"])
    mask, keep = kept(b.rng.tolist(), n * d, b.p)
    out = y + z * mask.cpu().view(n, d) * (65536 / keep)
    names = ("x", "w_in", "w_out", "norm_w", "weight")
    grads = dict(zip(names, torch.autograd.grad(out, [leaf[v] for v in names],
                                                b.dout.double().cpu())))
    # normwise: twelve stages, each a stored rounding and a sum of up to 1500 terms
    # whose roundings, in fp32, are within their number's root times 6 products
    lim = 12 * (half(b.t) + (6 * 1500) ** 0.5 * U)
    for got, ref, what in ((b.y, y, "y"), (b.out, out, "out"), (b.dx, grads["x"], "dx"),
                           (b.dw, grads["weight"], "dweight"), (b.dw_in, grads["w_in"], "dw_in"),
                           (b.dw_out, grads["w_out"], "dw_out"),
                           (b.dparams[1], grads["norm_w"], "dnorm")):
        err = float((got.double().cpu() - ref.detach()).norm() / ref.detach().norm())
        assert err <= lim, f"{what}: {err:.2e} of {lim:.2e}"


def test_block_on_another_stream_and_in_a_graph():
    b = Block(100, 136, 72, 4, 2, 0, torch.bfloat16, 0.2)
    b.run()
    torch.cuda.synchronize()
    want = {k: v.clone() for k, v in b.outputs().items()}

    def check(what):
        torch.cuda.synchronize()
        for k, v in b.outputs().items():
            assert torch.equal(v, want[k]), f"{what}: {k}"
            v.fill_(1)

    check("eager")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b.run(stream=side)
    check("another stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run()
    for i in range(3):
        b.ws.fill_(i * 100)
        graph.replay()
        check(f"replay {i}")
        assert float(b.x.float().sum()) == float(b.x.float().sum())
