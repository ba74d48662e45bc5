"""Attention whose scores pass what fp32 counts in ones: finite queries and
keys give finite outputs, those of the largest scores."""

import numpy as np
import pytest

import kv_model as km
import speculative_decoding_verification_amd as sv
from gpu_util import dev, host, torch

pytestmark = pytest.mark.gpu

KINDS = {"f16": km.F16, "bf16": km.BF16, "i8": km.I8}
U = 2.0 ** -24
# a scale that the conversion to base 2 takes to exactly 1: a score is q . k
# in base 2, without a rounding where the products and sums have none
ONE = float(np.float32(np.log(2)))
assert np.float32(np.float32(ONE) * np.float32(1.44269504088896340736)) == 1


def reference(q, k, v, n):
    """q [M, G, D], k and v [S, D] of one head: outputs in 64 bits, sums of
    weights times |v|, and the largest weight."""
    M, G, D = q.shape
    S = k.shape[0]
    out, mag, most = np.zeros((M, G, D)), np.zeros((M, G, D)), np.zeros((M, G, 1))
    for m in range(M):
        seen = S - n + m + 1
        for g in range(G):
            s = k[:seen].astype(np.float64) @ q[m, g].astype(np.float64) * ONE
            w = np.exp(s - s.max())
            w /= w.sum()
            out[m, g], mag[m, g], most[m, g] = w @ v[:seen], w @ np.abs(v[:seen]), w.max()
    return out, mag, most


def bound(mag, most, v, dim, slots, chunk):
    """The scores are whole numbers of fp32 and taken without rounding; what
    is left of attention_bound is the weights' exponents (differences of up
    to 64 in base 2 where a weight is not 0, off by half a step of the scale
    and of 2^x: below (3 dim + 16) u) and the sums.  Weights of far scores go
    up to 1, so that their two fp16 parts are off by 2^-25 of the largest."""
    return km.attention_bound(mag, np.ones(mag.shape[:2]), dim, slots, chunk) + slots * 2.0 ** -25 * most * np.abs(v).max(0)


class Filled:
    """One sequence of one key head: keys [S, D] and values, the last n of
    them the rows of the round."""

    def __init__(self, kind, k, v, n, group):
        S, D = k.shape
        self.n, self.group, self.D = n, group, D
        width = -(-S // 32)
        self.kv = sv.KvCache(kind, 1, 1, D, 32, width, 1, width)
        self.k, self.v = km.stored(k, kind), km.stored(v, kind)
        assert np.array_equal(self.k, k)   # the keys are exact in every type
        self.kv.reserve(S)
        self.kv.append(0, dev(k[None, :, None]), dev(v[None, :, None]))
        self.kv.lens.fill_(S - n)

    def run(self, q, chunk):
        out = torch().full((1, self.n, self.group, self.D), 77.0, device="cuda")
        self.kv.attention(self.group, 1, self.n, scale=ONE, chunk=chunk).run(0, dev(q[None]), out)
        return host(out)[0]

    def check(self, q, chunk):
        got = self.run(q, chunk)
        want, mag, most = reference(q, self.k, self.v, self.n)
        assert np.isfinite(got).all(), f"{np.isnan(got).sum()} NaN of {got.size}"
        limit = bound(mag, most, self.v, self.D, len(self.k), chunk)
        err = np.abs(got - want)
        assert (err <= limit).all(), (err / limit).max()


def keys(rng, first, D):
    """Keys of `first` in element 0 and small whole numbers in element 1;
    element 2, which no query reads, makes an int8 row's scale 1."""
    k = np.zeros((len(first), D), np.float32)
    k[:, 0] = first
    k[:, 1] = rng.integers(-8, 9, len(first))
    k[:, 2] = 127
    return k


def values(rng, kind, S, D):
    v = (rng.standard_normal((S, D)) * 2).astype(np.float32)
    if kind == "i8":  # scales far apart
        v *= (2.0 ** rng.integers(-12, 13, (S, 1))).astype(np.float32)
    return v


def queries(rng, n, group, D, power, key):
    """Scores of 2^power where element 0 of the key is `key`, a few of their
    steps apart."""
    q = np.zeros((n, group, D), np.float32)
    q[..., 0] = 2.0 ** power / key
    q[..., 1] = 2.0 ** max(0, power - 23)
    return q


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("power", [10, 22, 23, 24, 25, 26, 27, 28, 40, 100])
def test_large_scores(kind, sign, power):
    rng = np.random.default_rng(power)
    c = Filled(KINDS[kind], keys(rng, np.full(700, 64.0 * sign), 64), values(rng, kind, 700, 64), 3, 5)
    for chunk in (128, 1024):
        c.check(queries(rng, 3, 5, 64, power, 64), chunk)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("group,dim", [(20, 32), (20, 64), (20, 128), (3, 256)])
def test_large_scores_of_many_rows(kind, group, dim):
    """The same with several row tiles, and over head dimensions."""
    rng = np.random.default_rng(group + dim)
    c = Filled(KINDS[kind], keys(rng, np.full(300, 64.0), dim), values(rng, kind, 300, dim), 3, group)
    c.check(queries(rng, 3, group, dim, 25, 64), 512)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("order", ["up", "down", "mixed"])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_that_pass_the_border(kind, order, sign):
    """Scores of 2^21 to 2^27 in one row, so that the running maximum passes
    2^24 from either side."""
    rng = np.random.default_rng(7)
    first = np.sort(2.0 ** rng.integers(0, 7, 700))
    if order == "down":
        first = first[::-1]
    elif order == "mixed":
        first = rng.permutation(first)
    c = Filled(KINDS[kind], keys(rng, sign * first, 64), values(rng, kind, 700, 64), 3, 5)
    for chunk in (128, 1024):
        c.check(queries(rng, 3, 5, 64, 27, 64), chunk)


@pytest.mark.parametrize("kind", KINDS)
def test_rows_beside_large_scores(kind):
    """Rows of ordinary scores are the same bits whether or not the rows of
    their tile have scores past the border."""
    rng = np.random.default_rng(1)
    k = (rng.integers(-127, 128, (300, 64))).astype(np.float32)
    k[:, 2] = 127
    c = Filled(KINDS[kind], k, values(rng, kind, 300, 64), 3, 5)
    q = (rng.standard_normal((3, 5, 64)) / 64).astype(np.float32)
    for chunk in (128, 512):
        want = c.run(q, chunk)
        big = q.copy()
        big[1, ::2] *= np.float32(2.0 ** 30)
        big[2, 1] *= np.float32(2.0 ** 24)
        got = c.run(big, chunk)
        same = (big == q).all(-1)
        assert np.isfinite(got).all() and same.sum() == 11
        assert np.array_equal(got[same], want[same])


@pytest.mark.parametrize("power", [20, 25, 27, 40])
def test_large_scores_and_scales(power):
    """int8 rows whose values' scales are far apart as well: the weights with
    their scales are not bounded by the largest weight."""
    rng = np.random.default_rng(power)
    v = (rng.standard_normal((700, 64)) * 2.0 ** rng.integers(-60, 101, (700, 1))).astype(np.float32)
    c = Filled(km.I8, keys(rng, np.full(700, 64.0), 64), v, 3, 5)
    q = queries(rng, 3, 5, 64, power, 64)
    want, mag, _ = reference(q, c.k, c.v, 3)
    for chunk in (128, 1024):
        got = c.run(q, chunk)
        limit = km.attention_bound(mag, np.ones((3, 5)), 64, 700, chunk)
        if power < 24:  # two fp16 parts, 2^-39 of the largest weight with its scale (times a code) at worst
            limit = limit + 700 * 2.0 ** -39 * largest(q, c.k, c.v, 3)
        assert (np.abs(got - want) <= limit).all()


def largest(q, k, v, n):
    """The largest weight times the largest magnitude of its value's row."""
    top = np.abs(v.astype(np.float64)).max(-1)
    out = np.zeros(q.shape[:2] + (1,))
    for m in range(q.shape[0]):
        seen = len(k) - n + m + 1
        for g in range(q.shape[1]):
            s = k[:seen].astype(np.float64) @ q[m, g].astype(np.float64) * ONE
            w = np.exp(s - s.max())
            out[m, g] = (w / w.sum() * top[:seen]).max()
    return out


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("power", [100, 114, 115, 116, 117, 118, 120, 123, 126])
def test_very_large_queries(kind, power):
    """Queries up to the last power of two of fp32, whose scores still fit
    it: keys of -1, 0 and 1 in the element that is not 0."""
    rng = np.random.default_rng(power)
    for first in (rng.integers(-1, 2, 300), -np.ones(300)):
        k = np.zeros((300, 64), np.float32)
        k[:, 0], k[:, 2] = first, 127
        c = Filled(KINDS[kind], k, values(rng, kind, 300, 64), 3, 5)
        q = np.zeros((3, 5, 64), np.float32)
        q[..., 0] = 2.0 ** power
        q[0, 0, 1] = 2.0 ** (power - 30)
        for chunk in (128, 512):
            c.check(q, chunk)
