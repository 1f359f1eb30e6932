"""Inputs that show whether a product of fp32 values keeps all six products of their
bf16 parts, and the limit that a sum of them has to meet; on the CPU, where each of the
six is left out in turn.

An fp32 value is v = p0 + p1 + p2, each part the bf16 nearest to what is left.  Along k the
values of one operand come in pairs v, -p0(v), and those of the other are repeated: the
products of p0 cancel exactly, and a sum is made of the small products alone.  A product
of p2, or of p1 by p1, is about 2^-18 of one of first parts, and K / 2 independent ones
add up to 2^-18 (K / 2)^1/2 of it, about 30 K^1/2 U with U = 2^-24.

The limit: of the products that enter a sum, the K of first parts are the large ones.  What
they are added to holds a few that have not met their partners yet, 16 at most if a matrix
instruction took the even ones of its 32 k first, or 4 sizes of one.  An addition is
off by at most 2 U of that where it cuts, evenly spread, and K independent ones by
(8 / 3^1/2) K^1/2 U < 5 K^1/2 U.  The others are 2^-8 of these and vanish beside them."""
import pytest
import torch

U = 2.0 ** -24
SIX = [(2, 0), (0, 2), (1, 1), (1, 0), (0, 1), (0, 0)]


def limit(k):
    """Of the error's root mean square, by those of the operands' values."""
    return 5 * k ** 0.5 * U


def first_part(v):
    return v.to(torch.bfloat16).to(v.dtype)


def parts(v):
    out = []
    for _ in range(3):
        out.append(first_part(v))
        v = v - out[-1]
    return out


def paired(v, cancel):
    """Along the last dimension: v, -p0(v) or v, v; a last one without a partner is 0."""
    out, n = v.clone(), v.shape[-1] // 2 * 2
    even = out[..., 0:n:2]
    out[..., 1:n:2] = -first_part(even) if cancel else even
    out[..., n:] = 0
    return out


def rms(v):
    return float(v.double().pow(2).mean().sqrt())


def operands(side, m, n, k, seed):
    g = torch.Generator().manual_seed(seed)
    a, b = torch.randn(m, k, generator=g), torch.randn(n, k, generator=g)
    return paired(a, side == "first"), paired(b, side == "second")


def product(a, b, kinds):
    """Sum over k of the given products of parts, each exact, added in 64 bits."""
    pa, pb = ([p.double() for p in parts(v)] for v in (a, b))
    return sum(pa[i] @ pb[j].t() for i, j in kinds)


@pytest.mark.parametrize("k", [45, 136, 479, 900, 2500])
@pytest.mark.parametrize("side", ["first", "second"])
def test_a_lost_product_passes_the_limit(side, k):
    a, b = operands(side, 96, 80, k, k)
    assert all(torch.equal(sum(reversed(parts(v))), v) for v in (a, b)), "three parts are all"
    ref = a.double() @ b.double().t()
    lim = limit(k) * rms(a) * rms(b)
    assert rms(product(a, b, SIX) - ref) < 0.05 * lim
    seen = {"first": {(2, 0), (1, 1), (1, 0)}, "second": {(0, 2), (1, 1), (0, 1)}}[side]
    for lost in SIX:
        err = rms(product(a, b, [p for p in SIX if p != lost]) - ref)
        assert (err > 3 * lim) == (lost in seen), (lost, err / lim)


@pytest.mark.parametrize("side", ["first", "second"])
@pytest.mark.parametrize("even_first", [False, True])
def test_sums_in_fp32_meet_the_limit(side, even_first):
    """32 k at a time, the even ones of them first or as they come, every product of
    parts added for itself."""
    k = 480
    a, b = operands(side, 24, 20, k, 5)
    pa, pb = parts(a), parts(b)
    acc = torch.zeros(24, 20)
    for k0 in range(0, k, 32):
        order = list(range(k0, k0 + 32))
        if even_first:
            order = order[::2] + order[1::2]
        for i, j in SIX:
            for q in order:
                acc = acc + torch.outer(pa[i][:, q], pb[j][:, q])
    ref = a.double() @ b.double().t()
    assert rms(acc - ref) <= limit(k) * rms(a) * rms(b)


def test_what_the_six_leave_out_is_below_one_rounding():
    """|p1| <= 2^-8 and |p2| <= 2^-17 of a value's power of two."""
    g = torch.Generator().manual_seed(1)
    v = (1 + torch.rand(2, 1_000_000, generator=g)).clamp(max=2 - 2.0 ** -23)
    v[:, :1000] = 1 + 2.0 ** -8 + 2.0 ** -23 * torch.arange(-500, 500)
    (a0, a1, a2), (b0, b1, b2) = parts(v[0]), parts(v[1])
    assert max(float(p.abs().max()) for p in (a1, b1)) <= 2.0 ** -8
    assert max(float(p.abs().max()) for p in (a2, b2)) <= 2.0 ** -17
    a, b = v.double()
    left = sum(p.double() * q.double() for p, q in ((a1, b2), (a2, b1), (a2, b2)))
    assert float((left.abs() / (a * b)).max()) < U
