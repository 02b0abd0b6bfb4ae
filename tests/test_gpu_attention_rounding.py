"""Attention's probabilities keep more bits than its inputs' type.

Scores on two levels, so that the roundings of a level's probabilities do not
average out: a few tokens at the top, the others a distance below it, another
one for every head.

Tolerance.  A probability p goes into the product with the values as the sum of
two numbers of the inputs' type, hi and lo: hi is off by at most u p (u half a
step), and lo, which is p - hi exactly before it is rounded, by at most u |lo|,
so their sum by u^2 p; in fp16, where the largest p is 2^15, lo's step is never
less than 2^-24, so that n such terms add at most n 2^-40 of the largest value.
The rest is as for any inputs: scores off by e (their sum's roundings, dim + 4
of them, and 8 of their own size), the exponential by 2^-22, sums of n / 128 + 64
terms in fp32 above and below the fraction line, and half a step of the output.
Equal values c are given back as they are where that is less than half a step of
their own, which c = 1.9375 makes u / 1.9375 of c."""
import numpy as np
import pytest

import oracle
from tests import test_gpu_attention as base

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
f64 = base.f64


def levels(seed, lengths, D, page, x, cache=None, Hkv=2, G=16, deep=3.0):
    """A problem whose scores have two levels: every head's query is along the
    first element only, as are the keys; the levels' distance is the head's."""
    p = base.Problem(seed, lengths, Hkv * G, Hkv, D, page, x, cache, poison=False)
    k = torch.zeros(p.k.shape)
    k[..., 0] = -1.0
    k[:, ::5, :, 0] = 0.0
    keep = k.to(p.k.dtype)
    p.pools[0] = keep
    p.k.copy_(keep.to(p.k.device))
    q = torch.zeros(len(lengths), Hkv * G, D)
    q[..., 0] = deep * torch.rand(len(lengths), Hkv * G, generator=torch.Generator().manual_seed(seed + 1))
    p.q = q.to(base.T[x])
    p.dev[0].copy_(p.q.to(base.DEV))
    return p


def put_values(p, v):
    keep = v.to(p.v.dtype)
    p.pools[1] = keep
    p.v.copy_(keep.to(p.v.device))


def check(p, scale):
    out, lse = p.run(scale=scale)
    out = f64(out)
    u, two = torch.finfo(base.T[p.x]).eps / 2, 2.0 ** -40 if p.x == "f16" else 0.0
    for b, n in enumerate(p.lengths):
        pages = p.table[b].tolist()
        k, v = (oracle.paged(f64(t), pages, n) for t in p.pools)
        q = f64(p.q[b])
        want, _, z = oracle.attention(q, k, v, scale)
        for h in range(p.Hq):
            g = h // (p.Hq // p.Hkv)
            size = abs(scale) * (np.abs(k[:, g]) @ np.abs(q[h]))
            e = (p.D + 4) * U * size.max() + 8 * U * np.abs(z[h]).max()
            w = np.exp(z[h] - z[h].max())
            weight = w @ np.abs(v[:, g]) / w.sum()
            tol = (u * u + 2 * e + 2.0 ** -22 + 4 * (n / 128 + 64) * U) * weight + n * two * np.abs(v[:, g]).max() \
                + np.abs(want[h]) * u + U
            worst = (np.abs(out[b, h] - want[h]) - 1.01 * tol).max()
            assert worst <= 0, (b, n, h, worst, np.abs(out[b, h] - want[h]).max())


@pytest.mark.parametrize("x", ["f16", "bf16"])
@pytest.mark.parametrize("cache", [None, "e4m3"])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 24), (128, 64), (192, 16), (256, 16)])
def test_equal_values_come_back(x, cache, D, page):
    """The mean of equal values is that value, whatever the probabilities."""
    p = levels(D + page, [3, 40, 333, 1500], D, page, x, cache)
    c = 1.9375 if cache is None else 1.875   # of e4m3's 4 bits
    put_values(p, torch.full(p.v.shape, c))
    out, _ = p.run(scale=1.0)
    assert (f64(out) == c).all(), np.abs(f64(out) - c).max()


@pytest.mark.parametrize("x", ["f16", "bf16"])
@pytest.mark.parametrize("cache", [None, "e4m3"])
@pytest.mark.parametrize("deep", [1.0, 6.0, 14.0])
def test_probabilities_on_two_levels(x, cache, deep):
    """Values above zero, so that an error of a level is one of the output; a
    level may be all but nothing beside the other (e^-14)."""
    p = levels(int(deep), [7, 100, 2000], 128, 16, x, cache, deep=deep)
    g = torch.Generator().manual_seed(3)
    put_values(p, 0.5 + torch.rand(p.v.shape, generator=g))
    check(p, 1.0)


def test_a_long_tail():
    """Hundreds of thousands of tokens whose probabilities are small against one token's, and their sum is not."""
    for x in ("f16", "bf16"):
        p = levels(9, [200000], 64, 64, x, Hkv=1, G=4, deep=1.0)
        k = torch.zeros(p.k.shape)
        k[..., 0] = -1.0
        k[p.table[0, 0], 0, 0, 0] = 0.0
        p.pools[0] = k.to(p.k.dtype)
        p.k.copy_(p.pools[0].to(base.DEV))
        p.q[..., 0] = torch.tensor([11.0, 11.5, 12.0, 12.5]).to(p.q.dtype)
        p.dev[0].copy_(p.q.to(base.DEV))
        v = torch.full(p.v.shape, 1.0)
        v[p.table[0, 0], 0] = 0.0
        put_values(p, v)
        check(p, 1.0)


@pytest.mark.parametrize("x", ["f16", "bf16"])
def test_infinite_values_stay_infinite(x):
    """What is left off a probability may be zero or below; an infinite value of its token is no NaN for that, in a sequence
    of many pieces either.  Other elements of the head are off by one rounding of the probabilities at most (u of their
    weight, which is at most 1 here), other heads are as without it."""
    p = levels(21, [9000, 9000], 128, 64, x, Hkv=2, G=4, deep=2.0)
    g = torch.Generator().manual_seed(5)
    put_values(p, torch.rand(p.v.shape, generator=g))
    want = f64(p.run(scale=1.0)[0])
    pages, u = p.table[0].tolist(), torch.finfo(base.T[x]).eps / 2
    for token, element, value in ((3, 7, "inf"), (4444, 9, "-inf"), (8999, 127, "inf")):
        p.v[pages[token // 64], token % 64, 1, element] = float(value)
    got = f64(p.run(scale=1.0)[0])
    assert (got[1] == want[1]).all() and (got[0, :4] == want[0, :4]).all()
    assert (got[0, 4:, 7] == np.inf).all() and (got[0, 4:, 9] == -np.inf).all() and (got[0, 4:, 127] == np.inf).all()
    rest = np.delete(got[0, 4:], [7, 9, 127], axis=1), np.delete(want[0, 4:], [7, 9, 127], axis=1)
    assert (np.abs(rest[0] - rest[1]) <= 1.01 * u + 2 * u * np.abs(rest[1])).all()
    p.v[pages[70], 5, 1, 7] = float("-inf")   # both signs: NaN, as in the formula
    assert np.isnan(f64(p.run(scale=1.0)[0])[0, 4:, 7]).all()


def test_an_infinite_value_of_the_least_probability():
    """fp16's smallest probability is 2^-40 of the largest, and rounded from a little above half of that: an infinite value
    there is no NaN, one of a probability below is (0 times it), as with finite arithmetic of that type."""
    p = levels(30, [40], 64, 16, "f16", Hkv=1, G=4)
    put_values(p, torch.ones(p.v.shape))
    pages = p.table[0].tolist()
    k = torch.zeros(p.k.shape)
    k[..., 0] = -8.0                                  # all others vanish
    k[pages[0], 0, 0, 0] = 0.0
    k[pages[1], 1, 0, 0] = -1.0
    p.k.copy_(k.half().to(base.DEV))
    log2 = np.log(2.0)
    p.dev[0].zero_()
    p.dev[0][0, :, 0] = torch.tensor([39.2 * log2, 38.9 * log2, 30 * log2, log2]).half().to(base.DEV)
    p.v[pages[1], 1, 0, 3] = float("inf")
    out = f64(p.run(scale=1.0)[0])[0]
    assert (out[:, 3] == np.inf).all() and (np.delete(out, 3, axis=1) == 1).all(), out[:, 2:5]
