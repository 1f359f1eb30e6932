"""The expert block's operators against plain 64-bit forms of their formulas:
8-bit norm rows and their dispatch, dropout.

Tolerances are first-order error bounds counted from the formulas, with
U = 2^-24 the rounding of fp32 and half(t) that of the stored type."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

from recommender_embedding_tables_amd import embtab as eb  # noqa: E402
from tests.test_gpu_dense import (DEV, TYPES, U, gen, guarded, half, plain_sort, rand,  # noqa: E402
                                  within)

KINDS = list(TYPES)


# ---------------------------------------------------------------- norm to 8 bits

# A code's value before rounding is off by at most 127 * 42 U: squares and their
# sum of positive terms in 18 additions a row, halved by the root (13 U with the
# root's own 2 U), y's rounding there and in h (2 U), two products: h within 20 U,
# its maximum too, the quotient and the product by it 2 U more.
H_REL, CODE_ABS = 20 * U, 127 * 42 * U
NORM_SHAPES = [(1, 8), (3, 9), (5, 17), (130, 64), (7, 351), (33, 479), (64, 512), (3, 513),
               (17, 1000), (5, 2047), (9, 3328), (2, 8191), (3, 8192), (1500, 128), (4000, 24),
               (3600, 600)]


def add_norm(x, block, w, eps, y=None, shift=0):
    n, d = x.shape
    y2, check_y = guarded((n, d), x.dtype, shift=shift)
    y = y2 if y is None else y
    codes, check_c = guarded((n, d), torch.int8, shift=shift)
    scales, check_s = guarded((n,), torch.float32)
    eb.check(eb.emb_add_norm_int8(x, block, w, n, d, eb.dtype_code(x.dtype), eps, y, codes,
                                  scales), "add_norm_int8")
    torch.cuda.synchronize()
    for c in (check_y, check_c, check_s):
        c()
    return y, codes, scales


def norm_rows(seed, n, d, t, shift=0):
    g = gen(seed)
    x, block = (rand(g, n * d + shift, scale=s)[shift:].view(n, d) for s in (1.0, 0.5))
    x, block = (torch.empty(n * d + shift, dtype=t, device=DEV)[shift:].view(n, d).copy_(v)
                for v in (x, block))
    return x, block, 1 + 0.1 * rand(g, d)


def check_norm_rows(x, block, w, eps, y, codes, scales):
    ref = x.double() + block.double()
    within(y, ref, U * ref.abs(), "y")
    h = ref / torch.sqrt(ref.pow(2).mean(1, keepdim=True) + eps) * w.double()
    amax = h.abs().amax(1, keepdim=True)
    assert ((scales.double() - amax[:, 0] / 127).abs() <= (H_REL + 2 * U) * amax[:, 0] / 127 +
            2.0 ** -149).all()
    q = torch.where(amax > 0, h * 127 / amax, 0.0)
    off = (codes.double() - q).abs()
    assert (off <= 0.5 + CODE_ABS).all(), float(off.max())
    assert (codes.abs().amax(1)[amax[:, 0] > 0] == 127).all()


@pytest.mark.parametrize("n,d", NORM_SHAPES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shift", [0, 1])
def test_add_norm(n, d, kind, shift):
    x, block, w = norm_rows(n * 31 + d, n, d, TYPES[kind], shift)
    y, codes, scales = add_norm(x, block, w, 1e-6, shift=shift)
    check_norm_rows(x, block, w, 1e-6, y, codes, scales)
    again = add_norm(x, block, w, 1e-6)
    assert all(torch.equal(a, b) for a, b in zip(again, (y, codes, scales)))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,d", [(300, 33), (40, 1001), (9, 3327)])
def test_add_norm_in_place(n, d, kind):
    x, block, w = norm_rows(d, n, d, TYPES[kind])
    want = add_norm(x, block, w, 1e-5)
    for k in range(2):
        a, b = x.clone(), block.clone()
        got = add_norm(a, b, w, 1e-5, y=(a, b)[k])
        assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("scale", [1e-18, 1e-12, 1e12, 1e17])
def test_add_norm_of_rows_far_from_one(scale):
    x, block, w = norm_rows(5, 20, 200, torch.float32)
    x, block = x * scale, block * scale
    check_norm_rows(x, block, w, 0.0, *add_norm(x, block, w, 0.0))
    check_norm_rows(x, block, w, 1e-6, *add_norm(x, block, w, 1e-6))


def test_add_norm_of_tiny_weights_and_zero_rows():
    # |h| near 1e-37: 127 / amax would pass fp32's range
    x, block, w = norm_rows(6, 50, 96, torch.float32)
    w = w * 1e-37
    x[7] = block[7] = 0
    y, codes, scales = add_norm(x, block, w, 1e-6)
    check_norm_rows(x, block, w, 1e-6, y, codes, scales)
    assert (codes[7] == 0).all() and float(scales[7]) == 0
    y, codes, scales = add_norm(x, -x, w, 0.0)  # eps 0: the root of 0
    assert (y == 0).all()
    assert ((scales == 0) | scales.isnan()).all() and (codes == 0).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [40, 300, 2000, 3328])
def test_add_norm_of_rows_that_are_not_finite(kind, d):
    x, block, w = norm_rows(d, 30, d, TYPES[kind])
    want = add_norm(x, block, w, 1e-6)
    bad = {3: float("inf"), 11: float("nan"), 12: float("-inf"), 29: float("nan")}
    for r, v in bad.items():
        (x if r % 2 else block)[r, (r * 7) % d] = v
    y, codes, scales = add_norm(x, block, w, 1e-6)
    hit = torch.zeros(30, dtype=torch.bool, device=DEV)
    hit[list(bad)] = True
    assert scales[hit].isnan().all() and (codes[hit] == 0).all()
    for a, b in zip((y, codes, scales), want):
        assert torch.equal(a[~hit], b[~hit])


def test_add_norm_of_squares_beyond_the_range():
    x, block, w = norm_rows(8, 4, 64, torch.float32)
    x[2] = 1e25
    _, codes, scales = add_norm(x, block, w, 1e-6)
    assert scales.isnan().tolist() == [False, False, True, False] and (codes[2] == 0).all()


# ---------------------------------------------------------------- their dispatch

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,k,e,cap,d", [
    (1, 1, 1, 0, 8), (5, 2, 3, 0, 17), (64, 2, 8, 0, 512), (100, 3, 7, 30, 63), (300, 2, 16, 0, 479),
    (37, 4, 4, 64, 1000), (20, 1, 300, 2, 3328), (257, 8, 9, 0, 33), (11, 2, 5, 0, 4099)])
def test_dispatch_of_codes(n, k, e, cap, d, kind):
    r = np.random.default_rng(n * 3 + d)
    ids = np.stack([r.permutation(max(e, k))[:k] for _ in range(n)])
    ids[r.random(n) < 0.2] = -2
    ids[ids >= e] = -2
    _, src, pos = plain_sort(ids, e, cap)
    src, pos = (torch.from_numpy(np.ascontiguousarray(v)).to(DEV, torch.int32) for v in (src, pos))
    codes = torch.from_numpy(r.integers(-127, 128, n * d + 1, dtype=np.int8)).to(DEV)[1:].view(n, d)
    scales = torch.from_numpy(r.random(n).astype(np.float32) + 0.01).to(DEV)
    m = src.numel()
    xs, check = guarded((m, d), TYPES[kind], shift=1)
    eb.check(eb.emb_expert_dispatch_int8(codes, scales, pos, src, n, k, m, d,
                                         eb.dtype_code(xs.dtype), xs), "dispatch_int8")
    torch.cuda.synchronize()
    check()
    tok = torch.clamp(src.long(), min=0) // k
    ref = torch.where((src >= 0)[:, None], codes[tok].double() * scales[tok].double()[:, None], 0.0)
    within(xs, ref, U * ref.abs(), "xs")
    assert (xs[src < 0] == 0).all()


def test_rows_to_8_bits_and_back():
    n, d = 1000, 479
    x, block, w = norm_rows(1, n, d, torch.bfloat16)
    _, codes, scales = add_norm(x, block, w, 1e-6)
    place = torch.arange(n, dtype=torch.int32, device=DEV)
    back = torch.empty(n, d, device=DEV)
    eb.check(eb.emb_expert_dispatch_int8(codes, scales, place, place, n, 1, n, d, eb.EMB_F32,
                                         back), "dispatch_int8")
    assert torch.equal(back, codes.float() * scales[:, None])
    h = x.double() + block.double()
    h = h / torch.sqrt(h.pow(2).mean(1, keepdim=True) + 1e-6) * w.double()
    step = h.abs().amax(1, keepdim=True) / 127
    # half a step, the codes' own error and the value's rounding of |code| <= 127
    assert ((back.double() - h).abs() <= step * (0.5 + 2 * CODE_ABS + 127 * U)).all()


# ---------------------------------------------------------------- dropout

def sm64(v):
    with np.errstate(over="ignore"):
        z = v + np.uint64(0x9E3779B97F4A7C15)
        z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
        z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
        return z ^ (z >> np.uint64(31))


def kept(rng, n, p, first=0):
    """Which of the elements first .. first + n are kept (first a multiple of 4)."""
    seed, counter = (np.uint64(v & (2 ** 64 - 1)) for v in rng)
    with np.errstate(over="ignore"):
        group = counter + np.uint64(first // 4) + np.arange(-(-n // 4), dtype=np.uint64)
    h = sm64(sm64(np.array([seed])) ^ group)
    bits = np.stack([(h >> np.uint64(16 * j)) & np.uint64(0xFFFF) for j in range(4)], 1)
    keep = int(np.floor((1 - p) * 65536 + 0.5))
    return torch.from_numpy(bits.reshape(-1)[:n] < keep).to(DEV), keep


def dropout(x, res, p, rng, y=None, shift=0, stream=None):
    out, check = guarded((x.numel(),), x.dtype, shift=shift)
    y = out if y is None else y
    r = torch.tensor([((v + 2 ** 63) % 2 ** 64) - 2 ** 63 for v in rng], device=DEV)
    eb.check(eb.emb_dropout(x, res, x.numel(), eb.dtype_code(x.dtype), p, r, y, stream), "dropout")
    torch.cuda.synchronize()
    check()
    return y


def check_dropout(x, res, p, rng, y):
    mask, keep = kept(rng, x.numel(), p)
    branch = torch.where(mask, x.double() * (65536 / max(keep, 1)), 0.0)
    ref = branch + (res.double() if res is not None else 0.0)
    within(y, ref, U * (branch.abs() + ref.abs()), "y")
    if res is not None:
        assert torch.equal(y[~mask], res[~mask])
    else:
        assert (y[~mask] == 0).all()


NUMELS = [1, 2, 3, 4, 5, 7, 8, 9, 15, 1023, 1024, 1025, 2047, 2048, 2049, 100_003]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.999, 1.0, 2.0 ** -17])
@pytest.mark.parametrize("n", NUMELS)
def test_dropout(n, p, residual, kind):
    g, t, shift = gen(n), TYPES[kind], n % 3
    x, res = (rand(g, n + shift).to(t)[shift:] for _ in range(2))
    res = res if residual else None
    rng = (12345 + n, 7 * n)
    y = dropout(x, res, p, rng, shift=shift)
    check_dropout(x, res, p, rng, y)
    assert torch.equal(y, dropout(x, res, p, rng))
    if p in (0.0, 2.0 ** -17) and not residual:  # nothing is dropped: 2^-17 rounds to 0
        assert torch.equal(y, x)


@pytest.mark.parametrize("rng", [(0, 0), (-1, 2 ** 63 - 3), (2 ** 62 + 1, -2), (5, 2 ** 64 - 100)])
def test_dropout_of_any_seed_and_counter(rng):
    x = rand(gen(1), 10_000)
    y = dropout(x, None, 0.3, rng)
    check_dropout(x, None, 0.3, rng, y)
    share = float((y != 0).double().mean())
    assert abs(share - 0.7) <= 5 * (0.3 * 0.7 / 10_000) ** 0.5


def test_the_next_call_starts_past_this_ones_words():
    x = rand(gen(2), 1001)
    both = torch.cat([x[:400], x[400:]])
    whole = dropout(both, None, 0.4, (9, 100))
    parts = [dropout(both[:400], None, 0.4, (9, 100)),
             dropout(both[400:].clone(), None, 0.4, (9, 200))]
    assert torch.equal(whole, torch.cat(parts))


@pytest.mark.parametrize("kind", KINDS)
def test_dropout_in_place_and_of_values_that_are_not_finite(kind):
    g, t, n = gen(3), TYPES[kind], 5003
    x, res = rand(g, n).to(t), rand(g, n).to(t)
    want = dropout(x, res, 0.25, (3, 4))
    for k in range(2):
        a, b = x.clone(), res.clone()
        assert torch.equal(dropout(a, b, 0.25, (3, 4), y=(a, b)[k]), want)
    mask, _ = kept((3, 4), n, 0.25)
    x[~mask] = float("nan")
    x[torch.nonzero(~mask)[::2, 0]] = float("inf")
    assert torch.equal(dropout(x, res, 0.25, (3, 4)), want), "a dropped value counts for nothing"


def test_dropout_gradient_against_differences():
    n, rng = 300, (21, 22)
    g = gen(4)
    x, res, dy = (rand(g, n) for _ in range(3))
    dx = dropout(dy, None, 0.3, rng)
    for i in range(0, n, 17):
        e = torch.zeros(n, device=DEV)
        e[i] = 0.5
        up, down = (dropout(x + s * e, res, 0.3, rng).double() for s in (1, -1))
        slope = float(((up - down) * dy.double()).sum())
        # the two sides' roundings: of x +- e, the scale, the sum
        lim = 8 * U * float(dy[i].abs()) * (3 + 2 * float(x[i].abs()) + float(res[i].abs()))
        assert abs(slope - float(dx[i])) <= lim


def test_dropout_beyond_32_bit_indexes():
    n = 2 ** 32 + 1029
    x = torch.ones(n, dtype=torch.bfloat16, device=DEV)
    rng = torch.tensor([77, 5], device=DEV)
    eb.check(eb.emb_dropout(x, None, n, eb.EMB_BF16, 0.5, rng, x), "dropout")
    for first, count in ((0, 5000), (2 ** 31 - 4000, 8000), (2 ** 32 - 4000, 5029)):
        mask, _ = kept((77, 5), count, 0.5, first)
        assert torch.equal(x[first:first + count], torch.where(mask, 2.0, 0.0).bfloat16())


def test_small_operators_on_another_stream_and_in_a_graph():
    """Replays after the counter moved draw new words; eager work between them."""
    n, d = 64, 480
    x, block, w = norm_rows(3, n, d, torch.bfloat16)
    rng = torch.tensor([5, 1000], device=DEV)
    place = torch.arange(n, dtype=torch.int32, device=DEV)
    y, z, back = (torch.empty_like(x) for _ in range(3))
    codes, scales = torch.empty(n, d, dtype=torch.int8, device=DEV), torch.empty(n, device=DEV)

    def step():
        eb.check(eb.emb_add_norm_int8(x, block, w, n, d, eb.EMB_BF16, 1e-6, y, codes, scales), "n")
        eb.check(eb.emb_expert_dispatch_int8(codes, scales, place, place, n, 1, n, d, eb.EMB_BF16,
                                             back), "d")
        eb.check(eb.emb_dropout(back, y, n * d, eb.EMB_BF16, 0.3, rng, z), "o")
        rng[1] += n * d // 4

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    want = []
    for i in range(4):
        rng[1] = 1000 + i * (n * d // 4)
        step()
        want.append(z.clone())
    rng[1] = 1000
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    rng[1] = 1000
    for i in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(z, want[i]), i
        z.zero_()
        assert float((y.float() * 2).sum()) == float((y.float() * 2).sum())
    assert not torch.equal(want[0], want[1])
