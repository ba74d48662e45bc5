"""Attention at the end of the longest table row there can be."""

import numpy as np
import pytest

import kv_model as km
import speculative_decoding_verification_amd as sv
from gpu_util import dev, host, torch
from test_gpu_kv import ints, rows

pytestmark = pytest.mark.gpu

PAGE, DIM, M = 256, 32, 5
WIDTH = ((1 << 31) - 65536 - 1) // PAGE
LEN = WIDTH * PAGE - 40


@pytest.fixture(scope="module")
def cache():
    """2^31 - 65792 slots of which the first and the last page exist, 40 of
    the last one's not written yet; and its rows, without what lies between."""
    kv = sv.KvCache(km.I8, 1, 1, DIM, PAGE, 2, 1, WIDTH)
    kv.table[0, 0], kv.table[0, WIDTH - 1] = 0, 1
    rng = np.random.default_rng(0)
    parts = [rows(rng, 1, n, 1, DIM) for n in (PAGE, PAGE - 40, M)]
    for at, (k, v) in zip((0, LEN - (PAGE - 40), LEN), parts):
        kv.lens.fill_(at)
        kv.append(0, dev(k), dev(v))
    k, v = (np.concatenate([km.stored(p[i][0], km.I8) for p in parts]) for i in range(2))
    q = (rng.standard_normal((1, M, 3, DIM)) * 1.5).astype(np.float32)
    assert kv.status() == 0
    return kv, k, v, q


@pytest.mark.parametrize("window,sinks,chunk", [
    (64, 3, 0), (64, 3, 128), (64, 3, 8388096), (64, 3, 1 << 24), (200, 0, 4193920), (0, 0, 0), (0, 0, 2097024)])
def test_the_last_slots(cache, window, sinks, chunk):
    kv, k, v, q = cache
    out = torch().full((1, M, 3, DIM), 77.0, device="cuda")
    kv.attention(3, 1, M, window=window, sinks=sinks, chunk=chunk).run(0, dev(q), out)
    want, mag, amp = km.attention(q[0], k, v, 2 * PAGE - 40, M, DIM ** -0.5, window=window, sinks=sinks)
    # only these slots are summed, whatever the chunk
    assert (np.abs(host(out)[0] - want) <= km.attention_bound(mag, amp, DIM, 2 * PAGE, 1024)).all()


def test_the_row_is_full(cache):
    """The new rows past the end have no slot: 40 rows fit, the 41st does not."""
    kv, k, v, q = cache
    kv.lens.fill_(LEN + 40)
    out = torch().full((1, M, 3, DIM), 77.0, device="cuda")
    kv.attention(3, 1, M, window=1).run(0, dev(q), out)
    assert (host(out) == 0).all()
    kv.lens.fill_(LEN)
