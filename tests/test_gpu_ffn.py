"""The experts' gated feed-forward, forward and backward, against plain 64-bit
forms of its formulas.

Tolerances are first-order bounds counted from the formulas, with U = 2^-24 and
half(t) the rounding of the stored type.  A sum of K products is within
terms(K) * U of the sum of their magnitudes: every addition rounds once, by at
most 2 U where the matrix instruction cuts instead of rounding; an fp32 product
is six products of its parts, and what they leave out is below one U."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

from recommender_embedding_tables_amd import embtab as eb  # noqa: E402
from tests.test_gpu_dense import DEV, TINY, TYPES, U, gen, guarded, half, rand, within  # noqa: E402

ACTS = {"silu": eb.EMB_ACT_SILU, "gelu": eb.EMB_ACT_GELU, "relu": eb.EMB_ACT_RELU,
        "sigmoid": eb.EMB_ACT_SIGMOID}


def terms(k, t):
    return 2 * ((6 * k if t == torch.float32 else k) + 32)


def act64(act, v):
    """The activation and its slope in 64 bits."""
    if act == "relu":
        return v.clamp(min=0), (v > 0).double()
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-v / 2 ** 0.5)
        return v * cdf, cdf + v * torch.exp(-0.5 * v * v) / (2 * np.pi) ** 0.5
    s = torch.sigmoid(v)
    d = s * torch.sigmoid(-v)
    return (s, d) if act == "sigmoid" else (v * s, s + v * d)


# An activation's own error, relative to |act| + |v slope|: the exponential of a
# rounded argument (2 |v| + 4) U, a reciprocal or quotient, products: 16 U in all,
# erfc 16 U more.
def act_rel(v):
    return (32 + 4 * v.abs()) * U


class Case:
    """Inputs of one block; the rows of no expert hold NaN, outputs a marker there."""

    def __init__(self, counts, capacity, extra, dim, hidden, kind, act, seed=1, scale=1.0,
                 shift=0, dense=False):
        t = self.t = TYPES[kind]
        self.E, self.cap, self.D, self.F, self.act = len(counts), capacity, dim, hidden, act
        self.counts = counts
        starts = np.concatenate([[0], np.cumsum(counts)])
        self.M = M = capacity * self.E if capacity else int(starts[-1]) + extra
        self.groups = [(e * capacity if capacity else int(starts[e]), n)
                       for e, n in enumerate(counts)]
        self.offsets = None if dense else torch.tensor(starts, dtype=torch.int32, device=DEV)
        g = gen(seed)

        def values(*shape, s=1.0):
            n = int(np.prod(shape))
            x = torch.empty(n + shift, dtype=t, device=DEV)[shift:].view(shape)
            return x.copy_(rand(g, *shape, scale=s))

        self.live = torch.zeros(M, dtype=torch.bool, device=DEV)
        for r, n in self.groups:
            self.live[r:r + n] = True
        self.x, self.dy = values(M, dim, s=scale), values(M, dim)
        self.w_in = values(self.E, 2 * hidden, dim, s=dim ** -0.5)
        self.w_out = values(self.E, dim, hidden, s=hidden ** -0.5)
        self.gu = values(M, 2 * hidden, s=2 * scale)
        self.a = values(M, hidden)
        for v in (self.x, self.dy, self.gu, self.a):
            v[~self.live] = float("nan")
        self.code = eb.dtype_code(t)
        self.need = eb.emb_gated_ffn_workspace_bytes(M, self.E, dim, hidden, self.code)
        self.ws = torch.empty(self.need, dtype=torch.uint8, device=DEV).fill_(255)
        self.args = (M, self.E, capacity, dim, hidden, self.code, ACTS[act])

    def forward(self, keep=True, stream=None, shift=0):
        outs = [guarded(s, self.t, shift=shift)
                for s in ((self.M, 2 * self.F), (self.M, self.F), (self.M, self.D))]
        (gu, _), (a, _), (y, _) = outs
        eb.check(eb.emb_gated_ffn_forward(self.x, self.w_in, self.w_out, self.offsets, *self.args,
                                          gu if keep else None, a, y, self.ws, self.need, stream),
                 "forward")
        torch.cuda.synchronize()
        for v, check in outs:
            check()
            assert (v[~self.live] == 77).all(), "a row of no expert was written"
        return gu, a, y

    def backward(self, stream=None, shift=0):
        outs = [guarded(s, self.t, shift=shift)
                for s in ((self.M, self.D), self.w_in.shape, self.w_out.shape)]
        (dx, _), (dw_in, _), (dw_out, _) = outs
        eb.check(eb.emb_gated_ffn_backward(self.x, self.gu, self.a, self.w_in, self.w_out,
                                           self.dy, self.offsets, *self.args, dx, dw_in, dw_out,
                                           self.ws, self.need, stream), "backward")
        torch.cuda.synchronize()
        for _, check in outs:
            check()
        assert (dx[~self.live] == 77).all(), "a row of no expert was written"
        return dx, dw_in, dw_out

    def check_forward(self, gu, a, y):
        F, t = self.F, self.t
        for e, (r, n) in enumerate(self.groups):
            if n == 0:
                continue
            m = slice(r, r + n)
            x, w = self.x[m].double(), self.w_in[e].double()
            ref, size = x @ w.t(), x.abs() @ w.abs().t()
            off = terms(self.D, t) * U * size
            within(gu[m], ref, off, "gu")
            g, u = ref.split(F, 1)
            eg, eu = off.split(F, 1)
            f, slope = act64(self.act, g)
            # the slope changes by at most 1.2 times its argument's error
            eact = (slope.abs() + 1.2 * eg) * eg + act_rel(g) * (f.abs() + (g * slope).abs())
            within(a[m], f * u, eact * (u.abs() + eu) + f.abs() * eu + U * (f * u).abs(), "a")
            av, wo = a[m].double(), self.w_out[e].double()
            within(y[m], av @ wo.t(), terms(F, t) * U * (av.abs() @ wo.abs().t()), "y")

    def check_backward(self, dx, dw_in, dw_out):
        F, t = self.F, self.t
        for e, (r, n) in enumerate(self.groups):
            if n == 0:
                assert (dw_in[e] == 0).all() and (dw_out[e] == 0).all()
                continue
            m = slice(r, r + n)
            x, dy, a = (v[m].double() for v in (self.x, self.dy, self.a))
            w, wo = self.w_in[e].double(), self.w_out[e].double()
            g, u = self.gu[m].double().split(F, 1)
            within(dw_out[e], dy.t() @ a, terms(n, t) * U * (dy.abs().t() @ a.abs()), "dw_out")
            da, eda = dy @ wo, terms(self.D, t) * U * (dy.abs() @ wo.abs())
            f, slope = act64(self.act, g)
            ef = act_rel(g) * (f.abs() + (g * slope).abs())
            es = act_rel(g) * (1.2 + g.abs())  # slopes and what they are made of are below 1.2
            du, dg = da * f, da * u * slope
            edu = (da.abs() + eda) * ef + f.abs() * eda + 2 * U * du.abs()
            edg = u.abs() * ((da.abs() + eda) * es + slope.abs() * eda) + 3 * U * dg.abs()
            d, off = torch.cat([dg, du], 1), torch.cat([edg, edu], 1)
            if t != torch.float32:  # as stored between the products
                off = off + half(t) * (d.abs() + off) + TINY[t]
            size = d.abs() + off
            within(dx[m], d @ w, off @ w.abs() + terms(2 * F, t) * U * (size @ w.abs()), "dx")
            within(dw_in[e], d.t() @ x,
                   off.t() @ x.abs() + terms(n, t) * U * (size.t() @ x.abs()), "dw_in")


# counts, capacity, rows behind the last group, dim, hidden
SHAPES = [
    ([1], 0, 0, 8, 8),
    ([3, 0, 1], 0, 2, 9, 17),
    ([0, 5, 0, 20, 0], 0, 7, 33, 65),
    ([2, 1, 2, 3, 1, 4, 0, 3], 0, 0, 64, 96),
    ([16, 17, 15, 33], 0, 3, 128, 72),
    ([64, 129], 0, 1, 130, 100),
    ([127, 128, 0, 300], 0, 40, 64, 64),
    ([40, 3, 0, 100, 77], 100, 0, 72, 31),
    ([500], 0, 9, 479, 333),
    ([200, 313], 0, 0, 256, 512),
    ([700, 20], 0, 5, 96, 1000),
    ([5] * 70, 0, 0, 40, 24),
    ([7, 0, 2] * 300, 9, 0, 16, 8),
    ([1500], 0, 0, 136, 264),
    ([260, 515], 0, 0, 520, 392),
    ([0, 0], 0, 5, 16, 24),
]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_forward(shape, kind):
    c = Case(*SHAPES[shape], kind, "silu", seed=shape)
    gu, a, y = c.forward()
    c.check_forward(gu, a, y)
    _, a2, y2 = c.forward(keep=False)
    assert torch.equal(a2, a) and torch.equal(y2, y), "the same bits, gu kept or not"


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_backward(shape, kind):
    c = Case(*SHAPES[shape], kind, "silu", seed=50 + shape)
    got = c.backward()
    c.check_backward(*got)
    c.ws.fill_(7)
    assert all(torch.equal(p, q) for p, q in zip(c.backward(), got))


def ragged(experts, most, seed):
    """Group sizes 0 .. most, an empty one among them."""
    n = np.random.default_rng(seed).integers(0, most + 1, experts)
    n[experts // 2] = 0
    return [int(v) for v in n]


# Sizes at which the rules on sizes choose another kernel: large and small tiles of
# 16-bit values, whose widths end inside a slot, a half slot and a vector; parts of
# the weights' rows; fp32 in tiles of its own values and through planes, in blocks of
# 64 and 128 rows; one and more steps of experts in a wave.
PATHS = {
    "large": (ragged(20, 700, 1), 0, 3, 1032, 520),
    "large_half_slot": (ragged(20, 700, 2), 0, 0, 288, 1056),
    "large_odd_hidden": (ragged(20, 700, 3), 0, 1, 1032, 521),
    "large_odd_width": (ragged(20, 700, 4), 0, 0, 1031, 520),
    "large_capacity": (ragged(20, 400, 5), 400, 0, 776, 520),
    "parts": ([600 + i for i in range(17)], 0, 9, 264, 132),
    "tiles_fp32": ([900 - 3 * i for i in range(8)], 0, 5, 136, 520),
    "planes_64": ([900, 0, 37], 0, 0, 136, 333),
    "planes_128": ([1270], 0, 11, 72, 1400),
    "planes_128_backward": ([2500], 0, 0, 40, 1200),
    "experts_64": (ragged(64, 90, 6), 0, 2, 48, 40),
    "experts_65": (ragged(65, 90, 7), 0, 2, 48, 40),
}


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("path", list(PATHS))
def test_kernels_of_every_size(path, kind):
    c = Case(*PATHS[path], kind, "silu", seed=len(path))
    got = c.forward()
    c.check_forward(*got)
    assert all(torch.equal(p, q) for p, q in zip(c.forward(), got))
    got = c.backward()
    c.check_backward(*got)
    c.ws.fill_(7)
    assert all(torch.equal(p, q) for p, q in zip(c.backward(), got))


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("hidden", list(range(119, 131)) + [253, 254, 255])
def test_widths_at_the_end_of_a_tile(hidden, kind):
    c = Case([300], 0, 0, 40, hidden, kind, "silu", dense=True)
    c.check_forward(*c.forward())
    c.check_backward(*c.backward())
    c = Case([150, 70], 0, 0, hidden, 48, kind, "silu")
    c.check_forward(*c.forward())
    c.check_backward(*c.backward())


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("width", list(range(8, 34)) + list(range(248, 274)) + [513, 575, 767])
def test_few_rows_of_widths_that_end_inside_a_vector(width, kind):
    c = Case([3, 0, 19, 40], 0, 1, width, 2 * width - 7, kind, "silu")
    c.check_forward(*c.forward())


@pytest.mark.parametrize("dim,hidden", [(16_384, 65_528), (32_768, 32_768)])
def test_weights_of_two_gigabytes(dim, hidden):
    """Offsets of 32 bits just reach (the first) or do not (the second)."""
    t, rows = torch.bfloat16, 300
    g = gen(12)
    x = rand(g, rows, dim).to(t)
    w_in = torch.empty(1, 2 * hidden, dim, dtype=t, device=DEV)
    w_out = torch.empty(1, dim, hidden, dtype=t, device=DEV)
    for w, k in ((w_in, dim), (w_out, hidden)):
        for part in w[0].split(8192):
            part.copy_(rand(g, *part.shape, scale=k ** -0.5))
    gu, a, y = (torch.empty(rows, n, dtype=t, device=DEV) for n in (2 * hidden, hidden, dim))
    need = eb.emb_gated_ffn_workspace_bytes(rows, 1, dim, hidden, eb.EMB_BF16)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    args = (rows, 1, 0, dim, hidden, eb.EMB_BF16, eb.EMB_ACT_SILU)
    eb.check(eb.emb_gated_ffn_forward(x, w_in, w_out, None, *args, gu, a, y, ws, need), "forward")
    dx, dw_in, dw_out = torch.empty_like(x), torch.empty_like(w_in), torch.empty_like(w_out)
    eb.check(eb.emb_gated_ffn_backward(x, gu, a, w_in, w_out, y, None, *args, dx, dw_in, dw_out,
                                       ws, need), "backward")

    def product(p, q, what, got, k):
        p, q = p.double(), q.double()
        within(got, p @ q.t(), terms(k, t) * U * (p.abs() @ q.abs().t()), what)

    ends = [0, 1, hidden - 1, hidden, 2 * hidden - 1]
    product(x, w_in[0, ends], "gu", gu[:, ends], dim)
    product(a, w_out[0, [0, dim - 1]], "y", y[:, [0, dim - 1]], hidden)
    product(y.t()[[0, 7, dim - 1]], a.t(), "dw_out", dw_out[0, [0, 7, dim - 1]], rows)
    # dgu of the last unit, then its weights' gradients and its share of dx
    n = hidden - 1
    da = y.double() @ w_out[0, :, n].double()
    f, slope = act64("silu", gu[:, n].double())
    dg, du = da * gu[:, hidden + n].double() * slope, da * f
    for row, d in ((n, dg), (hidden + n, du)):
        ref = d @ x.double()
        err = float((dw_in[0, row].double() - ref).norm() / ref.norm())
        assert err <= 4 * half(t)  # dgu's rounding and the result's


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("scale", [0.3, 8.0])
def test_activations(act, scale, kind):
    c = Case([70, 0, 33], 0, 3, 64, 80, kind, act, scale=scale)
    c.check_forward(*c.forward())
    c.check_backward(*c.backward())


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("act", list(ACTS))
def test_activations_far_out(act, kind):
    """Gate pre-activations from 1e-3 to beyond the exponential's range, infinite and NaN,
    through the backward, whose da and u are 1: dw_in of one row is dgu itself."""
    t = TYPES[kind]
    top = 1e4 if kind == "f16" else 1e30
    far = torch.logspace(-3, np.log10(top), 118, dtype=torch.float64, device=DEV)
    near = torch.linspace(-20, 20, 81, dtype=torch.float64, device=DEV)
    g = torch.cat([far, -far, near, torch.tensor([float("inf"), float("-inf"), float("nan")],
                                                 dtype=torch.float64, device=DEV)])
    F = g.numel()
    c = Case([1], 0, 0, 8, F, kind, act)
    c.gu = torch.cat([g.to(t), torch.ones(F, dtype=t, device=DEV)]).view(1, -1)
    c.x.fill_(1.0)
    c.dy.fill_(0.0)
    c.dy[0, 0] = 1.0
    c.w_out.fill_(1.0)
    _, dw_in, _ = c.backward()
    got = dw_in[0, :, 0].double()
    f, slope = act64(act, c.gu[0, :F].double())
    lim = act_rel(c.gu[0, :F].double())
    ok = torch.isfinite(g)
    big = torch.finfo(t).max
    for name, v, ref in (("dg", got[:F], slope), ("du", got[F:], f)):
        r = ref[ok]
        # the slopes' parts are below 1.2; a slope 1 - s s' of a far gate may be off by them.
        # The hardware's exponential and reciprocal give 0 below 2^-126, which v (below
        # 104 where fp32 still holds e^v) makes |v| 2^-126 of v s and of its slope.
        v0 = c.gu[0, :F].double()[ok].abs().clamp(max=104)
        off = (lim[ok] * (r.abs() + (1.2 if name == "dg" else 0)) + 2 * half(t) * r.abs() + TINY[t]
               + (1 + v0) * 2.0 ** -126)
        assert ((v[ok] - r).abs() <= off)[r.abs() < big].all(), name
        assert v[-1].isnan() or act == "relu" and name == "dg", name
    if act == "sigmoid":
        assert got[F:][F - 3:F - 1].tolist() == [1.0, 0.0]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,dim,hidden", [(1, 64, 128), (300, 351, 100), (37, 8, 9),
                                             (1030, 256, 264)])
def test_dense_without_offsets(rows, dim, hidden, kind):
    c = Case([rows], 0, 0, dim, hidden, kind, "gelu", dense=True)
    c.check_forward(*c.forward())
    c.check_backward(*c.backward())


@pytest.mark.parametrize("kind", list(TYPES))
def test_operands_off_their_vectors_alignment(kind):
    for dim, hidden in ((64, 128), (256, 264), (67, 45)):
        c = Case([50, 200], 0, 3, dim, hidden, kind, "silu", shift=1)
        c.check_forward(*c.forward(shift=1))
        c.check_backward(*c.backward(shift=1))


@pytest.mark.parametrize("kind", list(TYPES))
def test_error_over_a_whole_matrix(kind):
    """Normwise: independent roundings add up as the root of their number."""
    c = Case([900], 0, 0, 479, 640, kind, "silu")
    gu, a, y = c.forward()
    x, w = c.x.double(), c.w_in[0].double()
    ref = x @ w.t()
    k = 6 * 479 if kind == "f32" else 479
    lim = k ** 0.5 * U + (half(c.t) if kind != "f32" else 0)
    assert float((gu.double() - ref).norm()) <= lim * float(ref.norm())
    dx, dw_in, dw_out = c.backward()
    ref = c.dy.double().t() @ c.a.double()
    k = 6 * 900 if kind == "f32" else 900
    lim = k ** 0.5 * U + (half(c.t) if kind != "f32" else 0)
    assert float((dw_out[0].double() - ref).norm()) <= lim * float(ref.norm())


@pytest.mark.parametrize("rows", [5, 300])
def test_subnormal_fp16_values_count(rows):
    """x near 3e-6 is below fp16's normal range, and its products are kept."""
    c = Case([rows], 0, 0, 264, 72, "f16", "silu", dense=True)
    c.x.mul_(3e-6)
    assert (c.x.float().abs() < 2.0 ** -14).all() and (c.x != 0).any()
    c.w_in.mul_(100)
    c.check_forward(*c.forward())
    gu = c.forward()[0].double()
    ref = c.x.double() @ c.w_in[0].double().t()
    assert float((gu - ref).norm()) <= 2 * half(torch.float16) * float(ref.norm()) + \
        2.0 ** -24 * gu.numel() ** 0.5


@pytest.mark.parametrize("act", list(ACTS))
def test_gradients_against_differences(act):
    """Of L = sum(y * dy) along a direction, beside what the difference itself is
    off in 64 bits."""
    c = Case([30, 11], 0, 0, 24, 40, "f32", act, seed=3)
    g = gen(9)
    gu, a, y = c.forward()
    c.gu, c.a = gu, a
    grads = dict(zip(("x", "w_in", "w_out"), c.backward()))
    h = 2.0 ** -6

    def loss64(x, w_in, w_out):
        total, size = 0.0, 0.0
        for e, (r, n) in enumerate(c.groups):
            m = slice(r, r + n)
            pre = x[m] @ w_in[e].t()
            y = (act64(act, pre[:, :c.F])[0] * pre[:, c.F:]) @ w_out[e].t()
            total = total + (y * c.dy[m].double()).sum()
            size = size + float((y.detach() * c.dy[m].double()).abs().sum())
        return total, size

    for name, grad in grads.items():
        base = {k: getattr(c, k) for k in ("x", "w_in", "w_out")}
        v = rand(g, *base[name].shape).sign()
        d64 = {k: w.double().requires_grad_() for k, w in base.items()}
        slope64 = float((torch.autograd.grad(loss64(**d64)[0], d64[name])[0] * v.double()).sum())
        ends, ends64 = [], []
        for s in (h, -h):
            moved = base[name] + s * v  # rounded: the 64-bit loss is of the same values
            setattr(c, name, moved)
            ends.append(float((c.forward()[2].double() * c.dy.double()).sum()))
            setattr(c, name, base[name])
            ends64.append(loss64(**{k: (moved if k == name else w).double()
                                    for k, w in base.items()}))
        slope = float((grad.double() * v.double()).sum())
        cut = abs((ends64[0][0] - ends64[1][0]) / (2 * h) - slope64)
        # y within the root of its operations' number of roundings, twice, over 2 h
        noise = 2 * (6 * 64 * 2) ** 0.5 * U * ends64[0][1] / (2 * h)
        assert abs((ends[0] - ends[1]) / (2 * h) - slope) <= float(cut) + noise + \
            1e-5 * abs(slope64), name
        assert abs(slope - slope64) <= 1e-5 * float((grad.double().abs()).sum()), name


@pytest.mark.parametrize("kind", list(TYPES))
def test_a_row_does_not_touch_another(kind):
    c = Case([40, 200, 3], 0, 2, 72, 88, kind, "silu")
    want = c.forward(), c.backward()
    for r in (5, 41, 242):
        for v in (c.x, c.gu, c.a, c.dy):
            v[r] = float("nan") if r % 2 else float("inf")
    got = c.forward(), c.backward()
    keep = torch.ones(c.M, dtype=torch.bool, device=DEV)
    keep[[5, 41, 242]] = False
    for p, q in zip(got[0] + got[1][:1], want[0] + want[1][:1]):
        assert torch.equal(p[keep & c.live], q[keep & c.live])
        assert not torch.isfinite(p[~keep].float()).all(1).any()


@pytest.mark.parametrize("offsets", [[0, 50, 20, 60], [-5, 3, 90, 2000], [0, 1000, 1000, 1001],
                                     [2000, 2100, 2200, 2300], [-2**31, 2**31 - 1, -1, 5]])
def test_offsets_that_name_no_rows_stay_inside_the_buffers(offsets):
    c = Case([20, 20, 20], 0, 4, 40, 48, "bf16", "silu")
    for v in (c.x, c.dy, c.gu, c.a):
        v.nan_to_num_(0.0)
    c.live[:] = True
    c.offsets = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    for run, shapes in ((c.forward, 3), (c.backward, 3)):
        live = c.live
        c.live = torch.ones_like(live)  # any row of the buffer may have been written
        assert len(run()) == shapes


def test_no_rows():
    c = Case([0, 0, 0], 0, 0, 24, 16, "bf16", "silu")
    assert c.M == 0
    c.forward()
    dx, dw_in, dw_out = c.backward()
    assert (dw_in == 0).all() and (dw_out == 0).all()


def test_indexes_beyond_32_bits():
    """2.2e9 pre-activations; the last rows against the plain form."""
    rows, D, F = 1_100_000, 64, 1024
    t = torch.bfloat16
    g = gen(4)
    x = rand(g, rows, D).to(t)
    w_in, w_out = (rand(g, 1, *s, scale=s[-1] ** -0.5).to(t) for s in ((2 * F, D), (D, F)))
    gu, a, y = (torch.empty(rows, n, dtype=t, device=DEV) for n in (2 * F, F, D))
    need = eb.emb_gated_ffn_workspace_bytes(rows, 1, D, F, eb.EMB_BF16)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    args = (rows, 1, 0, D, F, eb.EMB_BF16, eb.EMB_ACT_SILU)
    eb.check(eb.emb_gated_ffn_forward(x, w_in, w_out, None, *args, gu, a, y, ws, need), "forward")
    dx, dw_in, dw_out = torch.empty_like(x), torch.empty_like(w_in), torch.empty_like(w_out)
    eb.check(eb.emb_gated_ffn_backward(x, gu, a, w_in, w_out, y, None, *args, dx, dw_in, dw_out,
                                       ws, need), "backward")
    for r in (0, 1_048_500, rows - 100):
        c = Case([100], 0, 0, D, F, "bf16", "silu", dense=True)
        m = slice(r, r + 100)
        c.x, c.w_in, c.w_out, c.gu, c.a, c.dy = x[m], w_in, w_out, gu[m], a[m], y[m]
        c.check_forward(gu[m], a[m], y[m])
        sub = c.backward()
        assert torch.equal(sub[0], dx[m])
    ref = torch.zeros(D, F, dtype=torch.float64, device=DEV)
    size = torch.zeros_like(ref)
    for r in range(0, rows, 110_000):
        p, q = y[r:r + 110_000].double(), a[r:r + 110_000].double()
        ref += p.t() @ q
        size += p.abs().t() @ q.abs()
    within(dw_out[0], ref, terms(rows, t) * U * size, "dw_out")


def test_another_stream_and_a_graph_give_the_eager_bits():
    c = Case([100, 0, 300, 29], 0, 3, 128, 136, "bf16", "silu")
    d = Case([3, 9, 1], 0, 0, 128, 136, "bf16", "silu")  # few rows
    want = [c.forward(), c.backward(), d.forward()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [c.forward(stream=side), c.backward(stream=side), d.forward(stream=side)]
    for p, q in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(p, q))
    out = [torch.full_like(v, 77) for v in want[0] + want[1] + want[2]]

    def step():
        for k, at in ((c, 0), (d, 6)):
            eb.check(eb.emb_gated_ffn_forward(k.x, k.w_in, k.w_out, k.offsets, *k.args, out[at],
                                              out[at + 1], out[at + 2], k.ws, k.need), "f")
        eb.check(eb.emb_gated_ffn_backward(c.x, c.gu, c.a, c.w_in, c.w_out, c.dy, c.offsets,
                                           *c.args, out[3], out[4], out[5], c.ws, c.need), "b")

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for v in out:
            v.fill_(77)
        c.ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        for v, w in zip(out, want[0] + want[1] + want[2]):
            assert torch.equal(v, w)
        assert float(want[0][2][:5].float().sum()) == float(want[0][2][:5].float().sum())
