"""The expert training example: one step's loss, gradients, norm and updates
against automatic differentiation of the same model in 64 bits, and training
that lowers the loss."""
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

U = 2.0 ** -24
ROWS, DIM, BATCH = [3, 20, 300, 70], 16, 256


def plain_loss(m, p, x, labels, choice, pos):
    """The model from the lookup's rows x on, in 64 bits on the CPU."""
    def rms(v):
        return v / torch.sqrt((v * v).mean(1, keepdim=True) + ex.NORM_EPS)
    w = torch.softmax((x @ p["router"]).gather(1, choice), 1)
    block = torch.zeros_like(x)
    for j in range(m.topk):
        on = pos[:, j] >= 0  # beyond the expert's capacity: dropped
        rows = torch.einsum("nd,ndf->nf", x[on], p["experts"][choice[on, j]])
        block = block.index_add(0, torch.nonzero(on)[:, 0], w[on, j][:, None] * rows)
    a = torch.sigmoid(x @ p["gate"])[:, None]
    y = x + p["scale"] * a * (rms(block) * p["post"])
    logits = (rms(y) * p["pre"]) @ p["head"] + y.mean(1)
    return torch.nn.functional.binary_cross_entropy_with_logits(logits, labels)


def close(got, want, what):
    """Normwise: eight stages of sums of at most 256 terms, each within 256 U."""
    err = float((got.double().cpu() - want).norm())
    assert err <= 8 * 256 * U * float(want.norm()), f"{what}: {err / float(want.norm()):.2e}"


@pytest.mark.parametrize("max_norm", [1e9, 0.01])
def test_one_step_against_automatic_differentiation(max_norm):
    m = ex.Model(ROWS, DIM, BATCH, max_norm=max_norm)
    offsets, ids, labels = ex.batch_of(ROWS, BATCH, 5)
    p0 = {k: v.double().cpu().requires_grad_() for k, v in m.p.items()}
    w0 = m.tabs.weights.double().cpu().requires_grad_()
    acc0 = m.tabs.accum.double().cpu()
    loss, norm = m.step(offsets, ids, labels)
    torch.cuda.synchronize()
    starts = torch.tensor([sum(ROWS[:t]) for t in range(len(ROWS))])[:, None]
    row = ids.cpu().view(len(ROWS), BATCH) + starts
    x = w0[row].transpose(0, 1).reshape(BATCH, -1)
    assert torch.equal(m.x.double().cpu(), x.detach()), "one row per bag: the lookup is exact"
    want = plain_loss(m, p0, x, labels.double().cpu(), m.choice.cpu(), m.pos.cpu())
    assert (m.pos < 0).any() and (m.src < 0).any(), "some expert overflows and some row is empty"
    close(loss.view(1), want.detach().view(1), "loss")
    grads = torch.autograd.grad(want, list(p0.values()) + [w0])
    total = float(sum((g * g).sum() for g in grads)) ** 0.5
    coef = min(1.0, max_norm / (total + 1e-6))
    assert (coef < 1) == (max_norm < 1)
    close(norm, torch.tensor([total, coef], dtype=torch.float64), "norm")
    for k, g in zip(p0, grads):
        close(m.g[k], coef * g, "gradient of " + k)
        close(m.p[k], (p0[k] - m.lr * coef * g).detach(), k)
    g = coef * grads[-1]
    acc = acc0 + g * g
    close(m.tabs.accum, acc, "accumulators")
    step = m.lr * g / (acc.sqrt() + ex.ADAGRAD_EPS)
    close(m.tabs.weights, (w0 - step).detach(), "rows")
    m.close()


def test_training_lowers_the_loss():
    m = ex.Model(ROWS, DIM, BATCH, lr=0.1)
    batch = ex.batch_of(ROWS, BATCH, 9)
    losses = [float(m.step(*batch)[0]) for _ in range(40)]
    assert losses[-1] < 0.8 * losses[0], losses
    m.close()


def test_main_runs(capsys):
    losses = ex.main(["--steps", "3", "--batch", "512", "--dim", "16"])
    assert len(losses) == 3 and all(x == x for x in losses)
    assert capsys.readouterr().out.count("gradient norm") == 3
