"""The gated feed-forward in fp32 on inputs whose large products cancel in pairs, so that
its sums are made of the small products of the values' parts: every kernel and every
matrix product of both directions, against the limit of test_fp32_parts, which a sum
without any one of the six products passes by three times."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

from tests.test_fp32_parts import limit, paired  # noqa: E402
from tests.test_gpu_dense import DEV, gen, rand  # noqa: E402
from tests.test_gpu_ffn import Case, ragged  # noqa: E402

SIDES = ("first", "second")
# counts, capacity, rows behind the last group, dim, hidden: of the kernels that the rules
# on sizes choose.  Forward: few rows, tiles, planes in blocks of 64 and 128 rows (in the
# first and in the second product); backward: tiles, planes with rings of 4 and 2 stages
# and in blocks of 128 rows, the weights' rows whole and in parts.
SHAPES = {
    "few": ([3, 0, 19, 40], 0, 2, 479, 333),
    "few_dense": ([64], 0, 0, 1000, 136),
    "tiles": (ragged(64, 90, 6), 0, 2, 264, 520),
    "tiles_parts": ([900 - 3 * i for i in range(8)], 0, 5, 136, 520),
    "planes_64": ([900, 0, 37], 0, 0, 136, 333),
    "planes_capacity": ([300, 41, 0, 299], 300, 0, 479, 96),
    "planes_128_first": ([2500], 0, 11, 40, 1200),
    "planes_128_second": ([2500], 0, 0, 1400, 72),
}


def first_paired(v, cancel):
    """Pairs along the first dimension."""
    return paired(v.t().contiguous(), cancel).t().contiguous()


class Sums:
    """Root mean squares of errors and of the operands, over the groups."""

    def __init__(self):
        self.err = self.size = 0.0

    def add(self, got, a, b):
        """got = a b' with pairs along the last dimension of both."""
        a, b = a.double(), b.double()
        k = a.shape[-1]
        lim = limit(k) * float(a.pow(2).mean().sqrt() * b.pow(2).mean().sqrt())
        assert torch.isfinite(got).all()
        self.err += float((got.double() - a @ b.t()).pow(2).sum())
        self.size += lim ** 2 * got.numel()

    def check(self, what):
        assert 0 < self.size and self.err <= self.size, \
            f"{what}: {(self.err / self.size) ** 0.5:.3g} of the limit"


def places(n, d):
    """0, 1, .. below d, again from 0 where they end; pairs stay pairs."""
    return torch.arange(n, device=DEV) % (d // 2 * 2)


def one_hot(n, d):
    out = torch.zeros(n, d, device=DEV)
    out[torch.arange(n, device=DEV), places(n, d)] = 1
    return out


@pytest.mark.parametrize("side", SIDES)
@pytest.mark.parametrize("shape", list(SHAPES))
def test_pre_activations(shape, side):
    c = Case(*SHAPES[shape], "f32", "relu")
    c.x[c.live] = paired(c.x[c.live], side == "first")
    c.w_in.copy_(paired(c.w_in, side == "second"))
    gu = c.forward()[0]
    sums = Sums()
    for e, (r, n) in enumerate(c.groups):
        if n:
            sums.add(gu[r:r + n], c.x[r:r + n], c.w_in[e])
    sums.check("gu")


@pytest.mark.parametrize("side", SIDES)
@pytest.mark.parametrize("shape", list(SHAPES))
def test_output(shape, side):
    """x one value a row, the gate 0 and so act 1/2: a is half a column of Wu, exactly."""
    c = Case(*SHAPES[shape], "f32", "sigmoid")
    c.w_in[:, :c.F] = 0
    c.w_in[:, c.F:] = paired(rand(gen(2), c.E, c.D, c.F), side == "first").transpose(1, 2)
    c.w_out.copy_(paired(c.w_out, side == "second"))
    for r, n in c.groups:
        c.x[r:r + n] = one_hot(n, c.D)
    _, a, y = c.forward()
    sums = Sums()
    for e, (r, n) in enumerate(c.groups):
        if n:
            m = slice(r, r + n)
            assert torch.equal(a[m], 0.5 * c.w_in[e, c.F:, places(n, c.D)].t()), "exact values"
            sums.add(y[m], a[m], c.w_out[e])
    sums.check("y")


def backward_case(shape, **kw):
    """Gates and second pre-activations 1: both gradients of the pre-activations are da."""
    c = Case(*SHAPES[shape], "f32", "relu", **kw)
    c.gu[c.live] = 1
    return c


@pytest.mark.parametrize("side", SIDES)
@pytest.mark.parametrize("shape", list(SHAPES))
def test_gradient_of_the_second_weights(shape, side):
    c = backward_case(shape)
    for r, n in c.groups:
        if n:
            m = slice(r, r + n)
            c.dy[m] = first_paired(c.dy[m], side == "first")
            c.a[m] = first_paired(c.a[m], side == "second")
    dw_out = c.backward()[2]
    sums = Sums()
    for e, (r, n) in enumerate(c.groups):
        if n > 1:
            sums.add(dw_out[e], c.dy[r:r + n].t(), c.a[r:r + n].t())
    sums.check("dw_out")


@pytest.mark.parametrize("side", SIDES)
@pytest.mark.parametrize("shape", list(SHAPES))
def test_gradient_of_the_product(shape, side):
    """x one value a row: dw_in holds the pre-activations' gradients of the first rows."""
    c = backward_case(shape)
    c.dy[c.live] = paired(c.dy[c.live], side == "first")
    c.w_out.copy_(first_pairs_of_each(c.w_out, side == "second"))
    for r, n in c.groups:
        c.x[r:r + n] = 0
        k = min(n, c.D)
        c.x[r:r + k, :k] = torch.eye(k, device=DEV)
    dw_in = c.backward()[1]
    sums = Sums()
    for e, (r, n) in enumerate(c.groups):
        k = min(n, c.D)
        for half in dw_in[e, :, :k].split(c.F):
            if n:
                sums.add(half.t(), c.dy[r:r + k], c.w_out[e].t())
    sums.check("da")


def first_pairs_of_each(w, cancel):
    return torch.stack([first_paired(v, cancel) for v in w])


@pytest.mark.parametrize("side", SIDES)
@pytest.mark.parametrize("shape", list(SHAPES))
def test_gradient_of_the_input(shape, side):
    """dy one value a row: both gradients of the pre-activations are a row of Wo, exactly."""
    c = backward_case(shape)
    c.w_out.copy_(paired(c.w_out, side == "first"))
    for half in (slice(0, c.F), slice(c.F, 2 * c.F)):
        c.w_in[:, half] = first_pairs_of_each(c.w_in[:, half], side == "second")
    for r, n in c.groups:
        c.dy[r:r + n] = one_hot(n, c.D)
    dx = c.backward()[0]
    sums = Sums()
    for e, (r, n) in enumerate(c.groups):
        if n:
            d = c.w_out[e, places(n, c.D)]
            sums.add(dx[r:r + n], torch.cat([d, d], 1), c.w_in[e].t())
    sums.check("dx")


@pytest.mark.parametrize("side", SIDES)
@pytest.mark.parametrize("shape", list(SHAPES))
def test_gradient_of_the_first_weights(shape, side):
    c = backward_case(shape)
    c.w_out.copy_(first_pairs_of_each(c.w_out, side == "first"))
    for r, n in c.groups:
        if n:
            c.dy[r:r + n] = one_hot(n, c.D)
            c.x[r:r + n] = first_paired(c.x[r:r + n], side == "second")  # the odd one out is 0
    dw_in = c.backward()[1]
    sums = Sums()
    for e, (r, n) in enumerate(c.groups):
        if n > 1:
            d = c.w_out[e, places(n, c.D)]
            sums.add(dw_in[e], torch.cat([d, d], 1).t(), c.x[r:r + n].t())
    sums.check("dw_in")
