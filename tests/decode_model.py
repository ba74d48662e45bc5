"""Plain models of sampling with filters and of the residual's addition with
the RMS norm, written from their descriptions in 64 bits.  They share no code
with the GPU library."""

from __future__ import annotations

import numpy as np


def steps(V):
    """Bits of a weight's step: 2^-s with s = min(51, 63 - ceil(log2 V))."""
    return min(51, 63 - int(np.ceil(np.log2(V)))) if V > 1 else 51


def slack(V):
    """What a sum of V weights of at most 1 may be off by: half a step each,
    and a relative 2^-50 for each weight's exponential and its argument (both
    fp64 roundings, the argument at most 40 where the weight is no less than
    half a step: 40 * 2^-53 < 2^-47) of a sum of at most V."""
    return V * (2.0 ** -(steps(V) + 1) + 2.0 ** -46)


def order_of(z):
    """Indices by falling z, equal ones by rising index."""
    return np.lexsort((np.arange(z.size), -z.astype(np.float64)))


def weights(z, temperature):
    with np.errstate(over="ignore", invalid="ignore"):
        d = z.astype(np.float64) - float(z.max())
        return np.exp(d / temperature) if temperature > 0 else (d == 0).astype(np.float64)


def row_fails(z, params):
    t, k, p, m = params
    if not (0 <= t < np.inf and k >= 0 and 0 < p <= 1 and 0 <= m <= 1):
        return True
    return bool(np.isnan(z).any() or np.isposinf(z).any() or not np.isfinite(z).any())


def check_kept(z, keep, params):
    """Whether `keep` (truth values) is what the filters leave of a row, up to
    the roundings of the sums at a border."""
    t, k, p, m = params
    t, p, m = float(np.float32(t)), float(np.float32(p)), float(np.float32(m))
    if t == 0:
        t, k = 1.0, 1
    z = np.where(z == 0, np.float32(0), z)
    order = order_of(z)
    n = int(np.isfinite(z).sum())
    n = min(n, k) if k else n
    order = order[:n]
    w = weights(z, t)
    mass = np.cumsum(w[order])
    if p < 1:
        eps = slack(z.size)
        goal = p * mass[-1]
        least = int(np.searchsorted(mass, goal - eps)) + 1      # fewest that may be kept
        most = min(n, int(np.searchsorted(mass, goal + eps)) + 1)
    else:
        least = most = n
    # min-p cuts the run where the weights fall below it
    tell = 2.0 ** -45
    sure = int((w[order] >= m * (1 + tell)).sum())
    may = int((w[order] >= m * (1 - tell)).sum())
    got = int(keep.sum())
    assert min(least, sure) <= got <= min(most, may), (got, least, most, sure, may)
    want = np.zeros(z.size, bool)
    want[order[:got]] = True
    assert (keep == want).all()


def check_probs(z, keep, probs, temperature):
    w = weights(z, float(np.float32(temperature))) * keep
    want = w / w.sum()
    # the weight and the sum (fp64, above), and one rounding to fp32 (2^-24 of
    # the value, below 2^-126 half the least step 2^-149)
    tol = want * (2.0 ** -24 + 2 * slack(z.size) / w.sum() + 2.0 ** -45) + 2.0 ** -150
    assert (np.abs(probs - want) <= tol).all()


def check_token(z, keep, u, token, temperature):
    w = weights(z, float(np.float32(temperature))) * keep
    mass = np.cumsum(w)
    eps = slack(z.size)
    assert keep[token]
    assert mass[token] >= u * mass[-1] - 2 * eps
    assert mass[token] - w[token] <= u * mass[-1] + 2 * eps


def round_away(x):
    return np.sign(x) * np.floor(np.abs(x).astype(np.float64) + 0.5)


def codes(t, gamma):
    """The activation quantiser on fp32 t [rows, K]: codes, scales and sums,
    its roundings taken on fp32 values."""
    v = t if gamma is None else (t * gamma).astype(np.float32)
    b = v.reshape(t.shape[0], -1, 32)
    d = (np.abs(b).max(-1) / np.float32(127)).astype(np.float32)
    with np.errstate(divide="ignore"):
        inv = np.where(d != 0, np.float32(1) / d, np.float32(0)).astype(np.float32)
    q = np.clip(round_away((b * inv[..., None]).astype(np.float32)), -127, 127).astype(np.int8)
    return q.reshape(t.shape), d, q.reshape(t.shape[0], -1, 16).astype(np.int32).sum(-1)
