"""Commits of paths whose rows the cache never got."""

import numpy as np
import pytest

import kv_model as km
from gpu_util import dev
from test_gpu_kv import KINDS, Pair, ints, rows

pytestmark = pytest.mark.gpu


class Model(km.Model):
    """The model, where a path that names a row without a slot is refused
    like any other count that cannot be kept."""

    def commit(self, M, accepted, seq, n_new=None, path=None):
        if path is None:
            return super().commit(M, accepted, seq, n_new)
        # such a sequence is left as it was: a count that exceeds its rows
        # is what the plain bookkeeping refuses
        accepted = list(accepted)
        for b, s in self.first(seq):
            have = M if n_new is None else min(max(int(n_new[b]), 0), M)
            kept = int(accepted[b]) + 1
            if 0 < kept <= have and self.place(s, int(self.len[s]) + int(path[b][kept - 1])) is None:
                accepted[b] = M
        return super().commit(M, accepted, seq, n_new, path)


def pair(*args, **kw):
    p = Pair(*args, **kw)
    p.m.__class__ = Model
    return p


def round_of(p, rng, M, seq, acc, path, reserve=True):
    if reserve:
        p.kv.reserve(M, seq=ints(seq))
        p.m.reserve(M, seq)
    k, v = rows(rng, len(seq), M, p.m.heads, p.m.dim)
    for layer in range(p.kv.layers):
        p.kv.append(layer, dev(k), dev(v), seq=ints(seq))
    p.m.append(k, v, seq)
    p.kv.commit(M, ints(acc), seq=ints(seq), path=None if path is None else ints(path))
    p.m.commit(M, acc, seq, None, path)


@pytest.mark.parametrize("kind", KINDS)
def test_a_path_of_dropped_rows(kind):
    """60 slots in a page of 64 and none free: rows 4.. of the round are
    dropped.  A path that names one is refused and moves nothing, one of rows
    that were written is kept."""
    rng = np.random.default_rng(0)
    p = pair(KINDS[kind], 2, 64, 64, 1, 1, 3, layers=2)
    round_of(p, rng, 60, [0], [59], None)
    p.same()
    path = np.zeros((1, 16), np.int32)
    path[0, :2] = 0, 7
    before = p.kv.data.clone()
    round_of(p, rng, 16, [0], [1], path)
    assert p.m.len[0] == 60 and p.m.status == km.NO_PAGES | km.NO_SLOT | km.BAD_COMMIT
    p.same()
    p.same_rows(1)
    assert p.kv.status() == p.m.status
    p.m.status = 0
    # the committed rows are as they were, and row 1 of the round where append put it
    assert (p.kv.data != before).any()
    written = p.kv.data.clone()
    p.kv.commit(16, ints([1]), path=ints(path))
    assert (p.kv.data == written).all() and p.kv.status() == km.BAD_COMMIT
    path[0, :3] = 0, 2, 3
    round_of(p, rng, 16, [0], [2], path)
    assert p.m.len[0] == 63 and p.m.status == km.NO_PAGES | km.NO_SLOT
    p.same()
    for layer in range(2):
        p.same_rows(layer)


@pytest.mark.parametrize("width", [2, 3])
def test_a_path_past_the_table_row(width):
    """Rows past the end of the table row, with free pages left."""
    rng = np.random.default_rng(1)
    p = pair(km.F16, 1, 32, 32, 8, 1, width)
    round_of(p, rng, 32 * width - 3, [0], [32 * width - 4], None)
    path = np.zeros((1, 8), np.int32)
    path[0, :2] = 1, 3
    round_of(p, rng, 8, [0], [1], path)
    assert p.m.len[0] == 32 * width - 3 and p.m.status == km.TOO_LONG | km.NO_SLOT | km.BAD_COMMIT
    p.same()
    path[0, :2] = 1, 2
    round_of(p, rng, 8, [0], [1], path)
    assert p.m.len[0] == 32 * width - 1
    p.same()
    p.same_rows()


@pytest.mark.parametrize("kind,page,n_pages,seqs,width,seed", [
    ("f16", 32, 5, 3, 4, 0), ("i8", 64, 4, 4, 3, 1), ("bf16", 32, 7, 4, 3, 2)])
def test_random_paths_in_a_short_pool(kind, page, n_pages, seqs, width, seed):
    """Long random runs of rounds with paths in a pool that is nearly always
    full, some of them without a reservation."""
    rng = np.random.default_rng(seed)
    p = pair(KINDS[kind], 1, 32, page, n_pages, seqs, width)
    refused = 0
    for i in range(200):
        B, M = int(rng.integers(1, seqs + 1)), int(rng.integers(1, 17))
        seq = [int(x) for x in rng.permutation(seqs)[:B]]
        acc = [int(x) for x in rng.integers(-1, M, B)]
        path = np.zeros((B, M), np.int32)
        for b in range(B):
            path[b, :acc[b] + 1] = sorted(rng.permutation(M)[:acc[b] + 1])
        round_of(p, rng, M, seq, acc, path, reserve=rng.random() < 0.8)
        refused += bool(p.m.status & km.BAD_COMMIT)
        p.same()
        p.same_rows()
        assert p.kv.status() == p.m.status
        p.m.status = 0
        if len(p.m.free) == 0 and rng.random() < 0.3:
            s = [int(rng.integers(0, seqs))]
            p.kv.release(ints(s))
            p.m.release(s)
    assert refused > 10
