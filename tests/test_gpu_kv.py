"""The key-value cache on the GPU: rows in and out, the page operators
against the plain model, and attention against its definition in 64 bits."""

import numpy as np
import pytest

import kv_model as km
import speculative_decoding_verification_amd as sv
from gpu_util import dev, host, torch

pytestmark = pytest.mark.gpu

KINDS = {"f16": km.F16, "bf16": km.BF16, "i8": km.I8}


def ints(x):
    return dev(np.asarray(x, np.int32))


def rope_of(mode, rot, n_pos):
    if mode == 0:
        return None, (0, 0, None)
    t = sv.rope_table(n_pos, rot)
    return sv.Rope(mode, rot, t), (mode, rot, host(t))


class Pair:
    """A cache and its model, held in step."""

    def __init__(self, kind, heads, dim, page, n_pages, seqs, width, layers=1, fill=None):
        self.kv = sv.KvCache(kind, layers, heads, dim, page, n_pages, seqs, width)
        if fill is not None:
            self.kv.data.fill_(fill)
        self.m = km.Model(kind, heads, dim, page, n_pages, seqs, width)

    def same(self):
        kv, m = self.kv, self.m
        assert np.array_equal(host(kv.table), m.table)
        assert np.array_equal(host(kv.lens), m.len)
        assert np.array_equal(host(kv.refs), m.refs)
        ctl = host(kv.ctl)
        assert ctl[0] == len(m.free) and ctl[1] == m.status
        assert host(kv.free_ids)[:ctl[0]].tolist() == m.free

    def same_rows(self, layer=0, extra=0):
        """Every sequence's committed rows (and `extra` past them)."""
        kv, m = self.kv, self.m
        for s in range(m.seqs):
            n = int(m.len[s]) + extra
            if n == 0:
                continue
            k = torch().full((1, n, m.heads, m.dim), 7.0, device="cuda")
            v = k.clone()
            kv.read(layer, k, v, seq=ints([s]), start=ints([0]))
            wk, wv = m.read(s, 0, n)
            assert np.array_equal(host(k)[0], wk, equal_nan=True), (s, n)
            assert np.array_equal(host(v)[0], wv, equal_nan=True), (s, n)


def rows(rng, B, M, heads, dim):
    return [(rng.standard_normal((B, M, heads, dim)) * 2).astype(np.float32) for _ in "kv"]


# ------------------------------------------------------------ rows in, out
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads,dim,page,M,mode,rot", [
    (1, 32, 32, 1, 0, 0), (3, 96, 64, 5, 2, 96), (2, 128, 128, 70, 1, 64), (1, 256, 256, 300, 2, 128),
    (5, 160, 32, 33, 1, 6), (2, 64, 64, 16, 2, 10)])
def test_append_and_read(kind, heads, dim, page, M, mode, rot):
    rng = np.random.default_rng(dim + M)
    width = 4 + 700 // page
    p = Pair(KINDS[kind], heads, dim, page, 3 * width + 2, 3, width, layers=2, fill=0xFF)
    rope, mrope = rope_of(mode, rot, width * page)
    for lens in ([3, 0, page - 1], [31, page, 290]):
        p.kv.init()
        p.m = km.Model(KINDS[kind], heads, dim, page, 3 * width + 2, 3, width)
        p.m.len[:] = lens
        p.kv.lens.copy_(ints(lens))
        # pages of the committed slots too: reserved from an empty length
        for s, n in enumerate(lens):
            for obj in (p.kv, p.m):
                obj_len = obj.lens if obj is p.kv else obj.len
                obj_len[s] = 0
            if n:
                p.kv.reserve(n, seq=ints([s]))
                p.m.reserve(n, [s])
            p.kv.lens[s], p.m.len[s] = n, n
        p.kv.reserve(M)
        p.m.reserve(M, [0, 1, 2])
        p.same()
        k, v = rows(rng, 3, M, heads, dim)
        n_new = [M, max(1, M // 2), M - M // 3]
        p.kv.append(1, dev(k), dev(v), n_new=ints(n_new), rope=rope)
        p.m.append(k, v, [0, 1, 2], n_new, rope=mrope)
        for s in range(3):
            a = torch().full((1, M + 9, heads, dim), 5.0, device="cuda")
            b = a.clone()
            p.kv.read(1, a, b, seq=ints([s]), n_new=ints([n_new[s]]))
            wk, wv = p.m.read(s, lens[s], n_new[s])
            assert np.array_equal(host(a)[0, :n_new[s]], wk) and np.array_equal(host(b)[0, :n_new[s]], wv)
            assert (host(a)[0, n_new[s]:] == 5).all() and (host(b)[0, n_new[s]:] == 5).all()
        p.same()


@pytest.mark.parametrize("kind", KINDS)
def test_tree_rows_take_their_depths_positions(kind):
    p = Pair(KINDS[kind], 2, 64, 32, 8, 2, 4)
    rope, mrope = rope_of(2, 64, 128)
    rng = np.random.default_rng(1)
    tree = np.array([[1, 3, 5, 11, 0], [1, 2, 7, 9, 31]], np.int32)
    for s, n in ((0, 40), (1, 7)):
        p.kv.reserve(n, seq=ints([s]))
        p.m.reserve(n, [s])
        p.kv.lens[s], p.m.len[s] = n, n
    p.kv.reserve(5)
    p.m.reserve(5, [0, 1])
    k, v = rows(rng, 2, 5, 2, 64)
    p.kv.append(0, dev(k), dev(v), tree=ints(tree), rope=rope)
    p.m.append(k, v, [0, 1], tree=tree, rope=mrope)
    for s, n in ((0, 40), (1, 7)):
        a = torch().empty((1, 5, 2, 64), device="cuda")
        p.kv.read(0, a, seq=ints([s]))
        assert np.array_equal(host(a)[0], p.m.read(s, n, 5)[0])


@pytest.mark.parametrize("kind", KINDS)
def test_values_at_the_edges_of_the_types(kind):
    """Overflow, subnormals, ties, zeros, infinities and NaN as the type's
    rounding takes them; only the row that holds one is touched."""
    p = Pair(KINDS[kind], 1, 32, 32, 2, 1, 1)
    k = np.zeros((1, 8, 1, 32), np.float32)
    k[0, 0, 0, :6] = 65504, 65519.9, 65520, -70000, 6e-8, 2.0 ** -25
    k[0, 1, 0, :4] = 1 + 2.0 ** -11, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, -0.0
    k[0, 2, 0, :2] = np.inf, 1
    k[0, 3, 0, :2] = np.nan, 1
    k[0, 4] = 1e-39
    k[0, 5] = 3e38
    k[0, 6, 0, :4] = 127, 0.5, -0.5, 126.5
    v = k[:, ::-1].copy()
    p.kv.reserve(8)
    p.m.reserve(8, [0])
    p.kv.append(0, dev(k), dev(v))
    p.m.append(k, v, [0])
    a, b = (torch().empty((1, 8, 1, 32), device="cuda") for _ in "kv")
    p.kv.read(0, a, b)
    wk, wv = p.m.read(0, 0, 8)
    assert np.array_equal(host(a)[0], wk, equal_nan=True)
    assert np.array_equal(host(b)[0], wv, equal_nan=True)


def test_rows_without_a_page():
    """A row whose slot has no page is dropped and flagged; others and the
    pool stay whole.  Reads there give 0.  Sequences out of range have no
    rows, one named twice counts once."""
    p = Pair(km.F16, 1, 32, 32, 4, 3, 2)
    rng = np.random.default_rng(2)
    p.kv.reserve(32)
    p.m.reserve(32, [0, 1, 2])
    before = host(p.kv.data).copy()
    k, v = rows(rng, 3, 40, 1, 32)
    p.kv.append(0, dev(k), dev(v), n_new=ints([40, 0, -3]))
    p.m.append(k, v, [0, 1, 2], [40, 0, -3])
    assert p.m.status == km.NO_SLOT
    a = torch().full((1, 64, 1, 32), 9.0, device="cuda")
    p.kv.read(0, a, seq=ints([0]))
    assert np.array_equal(host(a)[0], p.m.read(0, 0, 64)[0]) and (host(a)[0, 32:] == 0).all()
    p.kv.read(0, a, seq=ints([0]), start=ints([-16]))
    assert (host(a)[0, :16] == 0).all() and np.array_equal(host(a)[0, 16:48], p.m.read(0, 0, 32)[0])
    for pages in (1, 2):
        after = host(p.kv.data).reshape(4, -1)[pages]
        assert np.array_equal(after, before.reshape(4, -1)[pages])
    assert p.kv.status() == km.NO_SLOT and p.kv.status() == 0
    p.m.status = 0
    k, v = rows(rng, 4, 2, 1, 32)
    seq = [2, 7, -1, 2]
    p.kv.append(0, dev(k), dev(v), seq=ints(seq))
    p.m.append(k, v, seq)
    p.kv.read(0, a[:, :2].contiguous(), seq=ints([2]))
    one = torch().empty((1, 2, 1, 32), device="cuda")
    p.kv.read(0, one, seq=ints([2]))
    assert np.array_equal(host(one)[0], p.m.read(2, 0, 2)[0])
    left = torch().full((2, 2, 1, 32), 3.0, device="cuda")
    p.kv.read(0, left, seq=ints([9, -5]))
    assert (host(left) == 3).all()
    # a table that names pages the pool does not have
    p.kv.table[1, 0] = 4
    p.kv.table[2, 0] = 1 << 30
    k, v = rows(rng, 3, 2, 1, 32)
    p.kv.append(0, dev(k), dev(v))
    assert p.kv.status() == km.NO_SLOT
    p.kv.read(0, left, seq=ints([1, 2]))
    assert (host(left) == 0).all()


# ------------------------------------------------------------- page calls
def step(p, rng, layers):
    """One random call on the cache and its model."""
    m, kv = p.m, p.kv
    B = int(rng.integers(1, m.seqs + 1))
    seq = [int(x) for x in rng.permutation(m.seqs)[:B]]
    if rng.random() < 0.2:
        seq[-1] = int(rng.integers(-1, m.seqs + 1))  # out of range, or named twice
    what = rng.choice(["round", "round", "round", "fork", "release", "compact", "reserve"])
    if what == "round":
        M = int(rng.integers(1, 17))
        n_new = [int(x) for x in rng.integers(0, M + 1, len(seq))] if rng.random() < 0.5 else None
        kv.reserve(M, seq=ints(seq), n_new=None if n_new is None else ints(n_new))
        m.reserve(M, seq, n_new)
        k, v = rows(rng, len(seq), M, m.heads, m.dim)
        for layer in range(layers):
            kv.append(layer, dev(k + layer), dev(v - layer), seq=ints(seq), n_new=None if n_new is None else ints(n_new))
        m.append(k + (layers - 1), v - (layers - 1), seq, n_new)
        have = [M] * len(seq) if n_new is None else n_new
        acc = [int(rng.integers(-1, h + 1)) for h in have]  # sometimes one too many
        path = None
        if rng.random() < 0.6:
            path = np.zeros((len(seq), M), np.int32)
            for b, h in enumerate(have):
                pick = sorted(rng.permutation(max(h, 1))[:acc[b] + 1])
                path[b, :len(pick)] = pick
                if rng.random() < 0.1 and M > 1:
                    path[b, 1] = path[b, 0]  # not ascending
        wide = np.full((len(seq), 3), 99, np.int32)
        wide[:, 0] = acc
        kv.commit(M, ints(wide), seq=ints(seq), n_new=None if n_new is None else ints(n_new),
                  path=None if path is None else ints(path))
        m.commit(M, acc, seq, n_new, path)
    elif what == "fork":
        empty = [s for s in range(m.seqs) if m.len[s] == 0 and m.table[s, 0] < 0]
        full = [s for s in range(m.seqs) if s not in empty]
        n = int(rng.integers(1, max(2, len(empty) + 1)))
        dst = (empty + full)[:n] if rng.random() < 0.85 else seq[:n]
        src = [int(rng.choice(full or [0])) for _ in dst]
        kv.fork(ints(src), ints(dst))
        m.fork(src, dst)
    elif what == "release":
        kv.release(ints(seq))
        m.release(seq)
    elif what == "compact":
        kv.compact()
        m.compact()
    else:
        n = int(rng.integers(1, 3 * m.page))
        kv.reserve(n, seq=ints(seq))
        m.reserve(n, seq)


@pytest.mark.parametrize("kind,heads,dim,page,n_pages,seqs,width,layers", [
    ("f16", 1, 32, 32, 24, 5, 6, 2), ("i8", 2, 64, 64, 40, 8, 5, 1), ("bf16", 1, 96, 32, 200, 40, 8, 1)])
def test_random_page_calls(kind, heads, dim, page, n_pages, seqs, width, layers):
    """Long random runs: tables, holders, free list in order, lengths, status
    and rows equal the model's after every call, and no page is lost."""
    rng = np.random.default_rng(n_pages)
    p = Pair(KINDS[kind], heads, dim, page, n_pages, seqs, width, layers)
    for i in range(150):
        step(p, rng, layers)
        p.same()
        held = [x for x in p.m.table.reshape(-1) if x >= 0]
        assert sorted(set(held)) == sorted(set(range(n_pages)) - set(p.m.free))
        if i % 10 == 9:
            p.same_rows(layers - 1)
            assert p.kv.status() == p.m.status
            p.m.status = 0
    p.kv.release(ints(range(seqs)))
    assert int(host(p.kv.ctl)[0]) == n_pages


def test_room_that_is_not_there():
    """Reservations and forks past the pool or the table row: all or nothing,
    flagged, and the next call starts clean."""
    p = Pair(km.F16, 1, 32, 32, 5, 4, 3)
    for n, seq, n_new, bits in ((40, [0, 1], None, 0), (20, [2, 3], None, km.NO_PAGES), (20, [2, 3], [20, 0], 0),
                                (100, [3], None, km.TOO_LONG), (97, [0, 3], [97, 1], km.TOO_LONG),
                                (1, [3], None, km.NO_PAGES)):
        p.kv.reserve(n, seq=ints(seq), n_new=None if n_new is None else ints(n_new))
        p.m.reserve(n, seq, n_new)
        assert p.m.status == bits
        p.same()
        assert p.kv.status() == bits
        p.m.status = 0
    p.kv.commit(40, ints([39, 39]), seq=ints([0, 1]))
    p.m.commit(40, [39, 39], [0, 1])
    p.kv.fork(ints([0]), ints([3]))
    p.m.fork([0], [3])
    assert p.m.status == km.NO_PAGES
    p.same()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("start", [0, 27, 63])
def test_long_paths(kind, start):
    """Paths of up to 31 of 32 rows: more than are moved at once, over block
    and page ends, in every layer."""
    p = Pair(KINDS[kind], 3, 96, 32, 20, 3, 6, layers=2)
    rng = np.random.default_rng(start)
    paths = [list(range(1, 32)), list(range(1, 32, 2)), [0, 1, 2, 5, 6, 7, 8, 9, 10, 20, 21, 22, 23, 30]]
    if start:
        k, v = rows(rng, 3, start, 3, 96)
        p.kv.reserve(start)
        p.m.reserve(start, [0, 1, 2])
        for layer in range(2):
            p.kv.append(layer, dev(k), dev(v))
        p.m.append(k, v, [0, 1, 2])
        p.kv.commit(start, ints([start - 1] * 3))
        p.m.commit(start, [start - 1] * 3, [0, 1, 2])
    k, v = rows(rng, 3, 32, 3, 96)
    p.kv.reserve(32)
    p.m.reserve(32, [0, 1, 2])
    for layer in range(2):
        p.kv.append(layer, dev(k), dev(v))
    p.m.append(k, v, [0, 1, 2])
    acc, path = [len(x) - 1 for x in paths], np.array([x + [0] * (32 - len(x)) for x in paths], np.int32)
    p.kv.commit(32, ints(acc), path=ints(path))
    p.m.commit(32, acc, [0, 1, 2], path=path)
    p.same()
    for layer in range(2):
        p.same_rows(layer)


@pytest.mark.parametrize("kind", KINDS)
def test_keys_or_values_alone(kind):
    kv = sv.KvCache(KINDS[kind], 1, 2, 64, 32, 4, 1, 4)
    k, v = rows(np.random.default_rng(1), 1, 50, 2, 64)
    kv.reserve(50)
    kv.append(0, dev(k), dev(v))
    both = [torch().zeros((1, 50, 2, 64), device="cuda") for _ in "kv"]
    kv.read(0, *both)
    for i in range(2):
        one = torch().zeros((1, 50, 2, 64), device="cuda")
        kv.read(0, **{("k_out", "v_out")[i]: one})
        assert np.array_equal(host(one), host(both[i])) and (host(one) != 0).any()


def test_pages_shared_and_copied():
    """Forks share the pages that are full and own a copy of the last one, in
    every layer; what one appends the others do not see; a shared page goes
    free with its last holder."""
    layers, p = 3, Pair(km.BF16, 2, 64, 64, 12, 4, 4, layers=3)
    rng = np.random.default_rng(5)
    p.kv.reserve(100, seq=ints([0]))
    p.m.reserve(100, [0])
    k, v = rows(rng, 1, 100, 2, 64)
    for layer in range(layers):
        p.kv.append(layer, dev(k + layer), dev(v), seq=ints([0]))
    p.m.append(k + 2, v, [0])
    p.kv.commit(100, ints([99]), seq=ints([0]))
    p.m.commit(100, [99], [0])
    p.kv.fork(ints([0, 0]), ints([2, 3]))
    p.m.fork([0, 0], [2, 3])
    p.same()
    p.same_rows(2)
    assert p.m.table[2, 0] == p.m.table[0, 0] and p.m.table[2, 1] != p.m.table[0, 1]
    k, v = rows(rng, 3, 40, 2, 64)
    p.kv.reserve(40, seq=ints([0, 2, 3]))
    p.m.reserve(40, [0, 2, 3])
    for layer in range(layers):
        p.kv.append(layer, dev(k + layer), dev(v), seq=ints([0, 2, 3]))
    p.m.append(k + 2, v, [0, 2, 3])
    p.kv.commit(40, ints([39, 39, 20]), seq=ints([0, 2, 3]))
    p.m.commit(40, [39, 39, 20], [0, 2, 3])
    p.same_rows(2)
    p.kv.release(ints([0, 3]))
    p.m.release([0, 3])
    p.same()
    p.same_rows(2)
    # more pairs than pages, a taken dst, a dst that is a src, a pair with itself: nothing happens
    for src, dst, bits in (([2] * 3, [0, 1, 1], km.BAD_FORK), ([2, 0], [0, 1], km.BAD_FORK), ([2], [2], km.BAD_FORK),
                           ([2, 5], [0, 1], km.BAD_FORK)):
        p.kv.fork(ints(src), ints(dst))
        assert p.kv.status() == bits
        p.same()


def test_a_pool_past_four_gib():
    """Blocks whose byte offset passes 2^32: written, read, attended to."""
    t = torch()
    heads, dim, page = 8, 128, 256
    n_pages = (9 << 29) // sv.kv_page_bytes(km.F16, heads, dim, page)
    kv = sv.KvCache(km.F16, 1, heads, dim, page, n_pages, 2, 4)
    kv.table[0, 0], kv.table[1, 0] = n_pages - 1, 0
    rng = np.random.default_rng(3)
    k, v = rows(rng, 2, 16, heads, dim)
    kv.append(0, dev(k), dev(v))
    a, b = (t.empty((2, 16, heads, dim), device="cuda") for _ in "kv")
    kv.read(0, a, b)
    assert np.array_equal(host(a), km.stored(k, km.F16)) and np.array_equal(host(b), km.stored(v, km.F16))
    q = rng.standard_normal((2, 16, heads, dim)).astype(np.float32)
    out = t.empty((2, 16, heads, dim), device="cuda")
    kv.attention(heads, 2, 16).run(0, dev(q), out)
    for s in range(2):
        want, mag, amp = km.attention(q[s], host(a)[s], host(b)[s], 0, 16, dim ** -0.5)
        assert (np.abs(host(out)[s] - want) <= km.attention_bound(mag, amp, dim, 16, 1024)).all()


# --------------------------------------------------------------- attention
class Case:
    """A cache filled with `lens` committed rows and n new ones each, and the
    reference's view of it."""

    def __init__(self, kind, heads, group, dim, page, lens, M, n_new=None, tree=None, window=0, sinks=0, mode=0, rot=0,
                 seed=0, fill=None, spare=2):
        self.rng = rng = np.random.default_rng(seed)
        self.kind, self.heads, self.group, self.dim, self.page = kind, heads, group, dim, page
        self.lens, self.M, self.window, self.sinks = lens, M, window, sinks
        B = self.B = len(lens)
        self.n_new = n_new if n_new is not None else [M] * B
        self.n_arg = None if n_new is None else ints(n_new)
        self.tree = tree
        width = -(-(max(lens) + M) // page)
        self.kv = kv = sv.KvCache(kind, 2, heads, dim, page, B * width + spare, B, width)
        kv.data.fill_(0xFF if fill is None else fill)  # every value a NaN where nothing is written
        order = rng.permutation(B * width + spare)[:B * width].reshape(B, width)
        kv.table.copy_(ints(order))
        self.rope, self.mrope = rope_of(mode, rot, width * page)
        self.k = np.zeros((B, width * page, heads, dim), np.float32)
        self.v = np.zeros_like(self.k)
        most = max(max(lens), 1)
        k, v = rows(rng, B, most, heads, dim)
        if any(lens):
            kv.append(1, dev(k), dev(v), n_new=ints(lens))
        kv.lens.copy_(ints(lens))
        nk, nv = rows(rng, B, M, heads, dim)
        kv.append(1, dev(nk), dev(nv), n_new=self.n_arg, tree=None if tree is None else ints(tree), rope=self.rope)
        for b in range(B):
            self.k[b, :lens[b]], self.v[b, :lens[b]] = km.stored(k[b, :lens[b]], kind), km.stored(v[b, :lens[b]], kind)
            masks = [(2 << m) - 1 for m in range(M)] if tree is None else tree[b]
            for m in range(self.n_new[b]):
                at = lens[b] + m
                self.k[b, at] = km.stored(km.rotated(nk[b, m], lens[b] + km.depth(masks, m), *self.mrope), kind)
                self.v[b, at] = km.stored(nv[b, m], kind)
        self.q = (rng.standard_normal((B, M, heads * group, dim)) * 1.5).astype(np.float32)
        self.scale = dim ** -0.5
        self.held = [np.ones(width * page, bool) for _ in range(B)]

    def run(self, out=None, chunk=0, ep=None, max_len=0, q=None, plan=None):
        if out is None:
            out = torch().full((self.B, self.M, self.heads * self.group, self.dim), 77.0, device="cuda")
        plan = plan or self.kv.attention(self.heads * self.group, self.B, self.M, scale=self.scale, window=self.window,
                                         sinks=self.sinks, chunk=chunk, max_len=max_len)
        plan.run(1, dev(self.q) if q is None else q, out, n_new=self.n_arg,
                 tree=None if self.tree is None else ints(self.tree), rope=self.rope, ep=ep)
        return host(out)

    def check(self, got, chunk=4096):
        for b in range(self.B):
            n = self.n_new[b]
            masks = [(2 << m) - 1 for m in range(self.M)] if self.tree is None else self.tree[b]
            q = np.stack([km.rotated(self.q[b, m], self.lens[b] + km.depth(masks, m), *self.mrope)
                          for m in range(self.M)])
            want, mag, amp = km.attention(q, self.k[b], self.v[b], self.lens[b], n, self.scale, self.held[b], masks,
                                          self.window, self.sinks)
            err = np.abs(got[b, :n] - want)
            slots = self.lens[b] + n
            assert (err <= km.attention_bound(mag, amp, self.dim, slots, chunk)).all(), (b, err.max())
            if np.linalg.norm(want):
                assert np.linalg.norm(err) / np.linalg.norm(want) <= km.norm_bound(amp, self.dim), b
            assert (got[b, n:] == 77).all()


TREE = np.array([[1, 3, 5, 11, 21, 0, 65, 128 + 21], [1, 2, 4, 8, 16, 32, 64, 255]], np.int32)

SHAPES = [  # kind, heads, group, dim, page, lens, M
    ("f16", 1, 1, 32, 32, [0], 1), ("f16", 2, 5, 128, 64, [1], 1), ("f16", 8, 5, 128, 64, [300], 5),
    ("bf16", 2, 4, 64, 32, [31, 32, 33, 95], 4), ("i8", 3, 2, 96, 128, [127, 128, 129], 16),
    ("i8", 2, 5, 128, 256, [1000, 17, 511], 5), ("bf16", 1, 64, 32, 64, [200], 3), ("f16", 2, 7, 160, 64, [257], 5),
    ("bf16", 2, 3, 192, 32, [400, 3], 6), ("i8", 1, 8, 224, 64, [130], 16), ("f16", 1, 16, 256, 128, [700, 5], 2),
    ("i8", 2, 1, 256, 64, [999], 1), ("bf16", 4, 8, 128, 64, [639, 2], 16), ("i8", 1, 3, 32, 32, [64, 63], 7),
    ("i8", 2, 2, 64, 64, [100], 9), ("i8", 1, 2, 160, 32, [77], 4), ("i8", 1, 1, 192, 32, [200], 16),
    ("bf16", 1, 1, 160, 32, [50], 16), ("bf16", 1, 2, 224, 32, [90], 9), ("bf16", 1, 1, 256, 32, [222], 16),
    ("f16", 1, 2, 64, 32, [90], 16), ("f16", 1, 2, 96, 32, [91], 9), ("f16", 1, 3, 192, 32, [92], 16),
    ("f16", 1, 3, 224, 256, [93], 16), ("bf16", 2, 2, 96, 64, [150, 1], 9)]


@pytest.mark.parametrize("kind,heads,group,dim,page,lens,M", SHAPES)
@pytest.mark.parametrize("chunk", [0, 128])
def test_attention(kind, heads, group, dim, page, lens, M, chunk):
    n_new = [1 + (M - 1) * (b % 2 == 0) for b in range(len(lens))] if len(lens) > 1 else None
    mode = (heads + M) % 3
    c = Case(KINDS[kind], heads, group, dim, page, lens, M, n_new=n_new, mode=mode, rot=dim // 2 if M % 2 else dim)
    c.check(c.run(chunk=chunk), chunk=chunk or 4096)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks,lens", [
    (1, 0, [5, 200]), (1, 3, [100, 0]), (7, 0, [40, 6]), (32, 4, [333, 31]), (100, 33, [500, 128]),
    (300, 1, [299, 900]), (64, 500, [450, 1200]), (5000, 2, [130, 700])])
def test_windows(kind, window, sinks, lens):
    c = Case(KINDS[kind], 2, 4, 64, 32, lens, 5, window=window, sinks=sinks, mode=2, rot=64)
    for chunk in (0, 128, 384):
        c.check(c.run(chunk=chunk), chunk=chunk or 4096)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (3, 0), (2, 1), (60, 33)])
def test_trees(kind, window, sinks):
    """Masks of trees, of rows that see nothing of the round, and of row 5 of
    the first sequence, which sees no new row at all."""
    c = Case(KINDS[kind], 2, 3, 128, 32, [61, 130], 8, tree=TREE, window=window, sinks=sinks, mode=1, rot=64)
    c.check(c.run(chunk=128), chunk=128)
    c.check(c.run())


def test_rows_that_see_nothing():
    """Rows that see no slot give zeros."""
    tree = np.array([[0, 0, 3], [1, 0, 4]], np.int32)
    c = Case(km.F16, 1, 2, 32, 32, [0, 0], 3, tree=tree)
    got = c.run()
    c.check(got)
    assert (got[0, :2] == 0).all() and (got[1, 1] == 0).all() and np.isfinite(got).all()
    c = Case(km.I8, 1, 2, 32, 32, [70, 40], 3, tree=tree, window=1)
    got = c.run(chunk=128)
    c.check(got)
    # row 2 sees rows 0 and 1, both at position 70, two before its own
    assert (got[0] == 0).all() and (got[1, 0] != 0).any()


@pytest.mark.parametrize("kind", ["f16", "bf16", "i8"])
def test_what_is_not_visible_changes_nothing(kind):
    """The same bits whatever hidden slots hold: NaN and infinities past the
    rows, before every window, in rows of the tree that a row does not see,
    and in other sequences' pages."""
    K = KINDS[kind]
    tree = np.array([[1, 3, 5, 1 + 8, 0, 32]], np.int32)
    for window, sinks in ((0, 0), (40, 5)):
        a = Case(K, 2, 3, 64, 32, [140], 6, tree=tree, window=window, sinks=sinks, seed=9, fill=0)
        b = Case(K, 2, 3, 64, 32, [140], 6, tree=tree, window=window, sinks=sinks, seed=9, fill=0xFF)
        want = a.run(chunk=128)
        assert np.array_equal(want, b.run(chunk=128)) and np.isfinite(want).all()
        a.check(want, chunk=128)
        # rows 1, 2, 3 see each other not at all: row 2's key and value not finite
        for bad in (np.inf, -np.inf, np.nan):
            k = torch().full((1, 1, 2, 64), 1.0, device="cuda")
            k[..., 5] = bad
            n = int(b.kv.lens[0])
            b.kv.lens[0] = n + 2
            b.kv.append(1, k, k)
            b.kv.lens[0] = n
            got = b.run(chunk=128)
            others = [0, 1, 3, 4, 5]
            assert np.array_equal(got[:, others], want[:, others])
            # row 2 sees itself: its outputs of that element are not finite
            assert not np.isfinite(got[0, 2, :, 5]).any()
        if window:  # slots between the sinks and the windows
            b = Case(K, 2, 3, 64, 32, [140], 6, tree=tree, window=window, sinks=sinks, seed=9, fill=0xFF)
            b.kv.lens[0] = 60
            bad = torch().full((1, 20, 2, 64), float("nan"), device="cuda")
            b.kv.append(1, bad, bad)
            b.kv.lens[0] = 140
            assert np.array_equal(b.run(chunk=128), want)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_a_value_that_is_not_finite_reaches_only_its_element(kind):
    """An infinite value in a committed slot that every row sees: its own
    element is infinite or NaN, and only in rows with a weight for it; in a
    window's edge the rows past it are untouched, bit for bit."""
    K = KINDS[kind]
    a, b = (Case(K, 1, 2, 64, 32, [90], 8, window=20, seed=4) for _ in "ab")
    want = a.run()
    # slot 74: inside the windows of rows at 90..93 (90 - 74 = 16 .. 19), outside those of 94..97
    b.kv.lens[0] = 74
    k = torch().zeros((1, 1, 1, 64), device="cuda")
    b.kv.read(1, k, start=ints([74]))
    v = dev(a.v[:, 74:75].copy())
    v[..., 7] = float("inf")
    b.kv.append(1, k, v)
    b.kv.lens[0] = 90
    got = b.run()
    assert np.array_equal(got[0, 4:], want[0, 4:])
    assert not np.isfinite(got[0, :4, :, 7]).any()
    rest = [i for i in range(64) if i != 7]
    assert np.array_equal(got[0, :4][..., rest], want[0, :4][..., rest])


@pytest.mark.parametrize("kind", KINDS)
def test_a_query_that_is_not_finite(kind):
    """A NaN or an infinity in q makes its own row's outputs NaN, with one
    chunk and with several, and no other's."""
    for B, group in ((1, 3), (8, 64)):
        c = Case(KINDS[kind], 2, group, 64, 32, [500] * B, 3)
        clean = {chunk: c.run(chunk=chunk) for chunk in (128, 1024)}
        c.q[0, 1, 2, 7], c.q[0, 2, 0, 3] = np.nan, np.inf
        for chunk, want in clean.items():
            got = c.run(chunk=chunk)
            assert np.isnan(got[0, 1, 2]).all() and np.isnan(got[0, 2, 0]).all()
            got[0, 1, 2], got[0, 2, 0] = want[0, 1, 2], want[0, 2, 0]
            assert np.array_equal(got, want)


def test_pages_that_are_not_there():
    """Entries of -1 or outside the pool: their slots are not visible."""
    for bad in (-1, 40, 1 << 30, -(1 << 31)):
        c = Case(km.BF16, 2, 2, 64, 32, [200, 90], 4, seed=2)
        c.kv.table[0, 2] = bad
        c.kv.table[1, 0] = bad
        c.held[0][64:96] = False
        c.held[1][:32] = False
        c.check(c.run(chunk=128), chunk=128)
    c = Case(km.F16, 1, 1, 32, 32, [40], 2)
    c.kv.table.fill_(-1)
    assert (c.run() == 0).all()


def test_sequences_of_a_call():
    """A list of sequences in any order, twice the same, out of range; M that
    some rows do not use; lengths out of range are held within the table."""
    t = torch()
    c = Case(km.F16, 2, 2, 64, 32, [10, 70, 33], 3, seed=1)
    want = c.run()
    plan = c.kv.attention(4, 5, 3)
    out = t.full((5, 3, 4, 64), 77.0, device="cuda")
    q = np.concatenate([c.q[2:], c.q[:1], c.q[:1], c.q[:1], c.q[2:]])
    plan.run(1, dev(q), out, seq=ints([2, 0, -1, 3, 2]))
    got = host(out)
    assert np.array_equal(got[0], want[2]) and np.array_equal(got[1], want[0]) and np.array_equal(got[4], want[2])
    assert (got[2:4] == 77).all()
    out.fill_(77.0)
    plan.run(1, dev(q), out, seq=ints([2, 0, 1, 0, 2]), n_new=ints([0, -1, 0, 99, 0]))
    got = host(out)
    assert (got[[0, 1, 2, 4]] == 77).all() and np.array_equal(got[3], want[0])
    for n, held in ((-5, 0), (1 << 30, 96)):  # three pages of 32 slots; those past the rows hold NaN
        c.kv.lens[1] = n
        got = c.run()
        c.kv.lens[1] = held
        assert np.array_equal(got, c.run(), equal_nan=True) and np.isfinite(got[[0, 2]]).all()


def test_longer_than_max_len():
    c = Case(km.F16, 2, 2, 64, 32, [10, 700, 300], 3, seed=1)
    want = c.run(chunk=128)
    got = c.run(max_len=303, chunk=128)
    assert np.isnan(got[1]).all() and np.array_equal(got[[0, 2]], want[[0, 2]])
    assert c.kv.status() == km.OVER_MAX
    got = c.run(max_len=100, chunk=128)   # one chunk: no join
    assert np.isnan(got[1:]).all() and np.array_equal(got[0], want[0])
    assert c.kv.status() == km.OVER_MAX
    assert np.array_equal(c.run(max_len=703, chunk=128), want) and c.kv.status() == 0


@pytest.mark.parametrize("kind,window,sinks,tree", [
    ("f16", 0, 0, False), ("bf16", 37, 3, False), ("i8", 0, 0, False), ("f16", 50, 70, True), ("i8", 129, 0, True),
    ("bf16", 0, 0, True)])
@pytest.mark.parametrize("group,dim", [(5, 128), (3, 64), (2, 192)])
def test_a_row_does_not_depend_on_the_others(kind, window, sinks, tree, group, dim):
    """Row m of a round equals, bit for bit, the row run alone over a cache
    that already holds the rows before it, and does not depend on the other
    sequences of the call."""
    t = torch()
    masks = np.tile(np.array([[1, 3, 7, 15, 31, 63, 127]], np.int32), (2, 1)) if tree else None
    c = Case(KINDS[kind], 2, group, dim, 32, [253, 380], 7, tree=masks, window=window, sinks=sinks, mode=2, rot=dim)
    want = c.run(chunk=128)
    c.check(want, chunk=128)
    for m in range(7):
        for b in range(2):
            c.kv.lens.copy_(ints(c.lens))
            c.kv.lens[b] += m
            plan = c.kv.attention(2 * group, 1, 1, scale=c.scale, window=window, sinks=sinks, chunk=128)
            out = t.empty((1, 1, 2 * group, dim), device="cuda")
            plan.run(1, dev(c.q[b:b + 1, m:m + 1].copy()), out, seq=ints([b]), rope=c.rope)
            assert np.array_equal(host(out)[0, 0], want[b, m]), (m, b)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads,group,dim,M,mode,rot", [
    (1, 3, 32, 16, 2, 24), (2, 4, 64, 16, 1, 64), (1, 5, 96, 5, 2, 20), (2, 5, 128, 5, 2, 128), (1, 2, 160, 9, 1, 160),
    (1, 3, 192, 4, 2, 96), (1, 1, 224, 16, 1, 6), (1, 16, 256, 1, 2, 256)])
def test_long_chunks(kind, heads, group, dim, M, mode, rot):
    """Chunks of more than 512 slots, one and several a sequence."""
    c = Case(KINDS[kind], heads, group, dim, 32, [1300, 611], M, mode=mode, rot=rot)
    c.check(c.run(chunk=640), chunk=640)
    c.check(c.run(chunk=2048), chunk=2048)


@pytest.mark.parametrize("kind,window,sinks", [("f16", 0, 0), ("bf16", 700, 40), ("i8", 1100, 700)])
def test_a_row_of_many_and_long_chunks(kind, window, sinks):
    """A row's bits with as many rows as fit (which are joined by threads of
    their own) and alone, in chunks of more than 512 slots."""
    t = torch()
    c = Case(KINDS[kind], 4, 8, 128, 32, [2900, 700, 1300, 640, 3, 1281, 2200], 16, window=window, sinks=sinks, mode=2,
             rot=128)
    for chunk in (128, 640):
        want = c.run(chunk=chunk)
        c.check(want, chunk=chunk)
        for b in range(7):
            for m in (0, 9, 15):
                c.kv.lens.copy_(ints(c.lens))
                c.kv.lens[b] += m
                plan = c.kv.attention(32, 1, 1, scale=c.scale, window=window, sinks=sinks, chunk=chunk)
                out = t.empty((1, 1, 32, 128), device="cuda")
                plan.run(1, dev(c.q[b:b + 1, m:m + 1].copy()), out, seq=ints([b]), rope=c.rope)
                assert np.array_equal(host(out)[0, 0], want[b, m]), (chunk, m, b)
        c.kv.lens.copy_(ints(c.lens))


@pytest.mark.parametrize("kind,window,sinks", [("f16", 0, 0), ("i8", 150, 9)])
def test_many_sequences(kind, window, sinks):
    """More sequences than a wave has lanes, of lengths from 0 on, one of them
    named twice and one out of range."""
    rng = np.random.default_rng(4)
    lens = [int(n) for n in rng.integers(0, 700, 150)]
    lens[3] = lens[77] = 0
    c = Case(KINDS[kind], 2, 2, 32, 64, lens, 2, n_new=[1 + b % 2 for b in range(150)], window=window, sinks=sinks)
    for chunk in (0, 128):
        got = c.run(chunk=chunk)
        c.check(got, chunk=chunk or 4096)
    seq = [149, 20, 20, 150, 64] + list(range(70))
    plan = c.kv.attention(4, len(seq), 2, scale=c.scale, window=window, sinks=sinks, chunk=128)
    q = np.stack([c.q[min(s, 149)] for s in seq])
    out = torch().full((len(seq), 2, 4, 32), 77.0, device="cuda")
    plan.run(1, dev(q), out, seq=ints(seq), n_new=ints([1 + s % 2 for s in seq]))
    for i, s in enumerate(seq):
        want = np.full((2, 4, 32), 77, np.float32) if s == 150 else got[s]
        assert np.array_equal(host(out)[i], want), (i, s)


def test_more_chunks_than_a_join_holds():
    """1094 chunks, whose weights pass the join's table."""
    c = Case(km.F16, 1, 2, 32, 256, [140000, 139900], 1, seed=5)
    c.check(c.run(chunk=128), chunk=128)


@pytest.mark.parametrize("lens,chunk", [([300, 20], 128), ([60, 20], 0)])
@pytest.mark.parametrize("gamma", [False, True])
def test_requantised_output(lens, chunk, gamma):
    """The epilogue's codes, scales, code sums and partials are those that
    sv_quantize_act_q8 makes of out, alone and beside out; rows not in use
    stay as they were."""
    t = torch()
    c = Case(km.BF16, 2, 3, 96, 32, lens, 4, n_new=[4, 2])
    K = 6 * 96
    g = dev((1 + 0.1 * np.random.default_rng(0).standard_normal(K)).astype(np.float32)) if gamma else None

    def act():
        return (t.full((8, K), 9, dtype=t.int8, device="cuda"), t.full((8, K // 32), 9.0, device="cuda"),
                t.full((8, K // 16), 9, dtype=t.int32, device="cuda"), t.full((8, K // 32), 9.0, device="cuda"))

    want, both, only = act(), act(), act()
    out = t.zeros((2, 4, 6, 96), device="cuda")
    c.run(out, chunk=chunk)
    sv.quantize_act_q8(out.view(8, K), want[0], want[1], want[2], gamma=g, sumsq=want[3])
    beside = t.zeros_like(out)
    c.run(beside, chunk=chunk, ep=sv.epilogue(sv.SV_EP_QUANT, *both, gamma=g))
    assert np.array_equal(host(out), host(beside))
    plan = c.kv.attention(6, 2, 4, chunk=chunk)
    plan.run(1, dev(c.q), None, n_new=c.n_arg, ep=sv.epilogue(sv.SV_EP_QUANT, *only, gamma=g))
    live = [0, 1, 2, 3, 4, 5]
    for w, x, y in zip(want, both, only):
        assert np.array_equal(host(w)[live], host(x)[live]) and np.array_equal(host(w)[live], host(y)[live])
        assert (host(x)[6:] == 9).all() and (host(y)[6:] == 9).all()


def test_far_positions_and_long_lengths():
    """40000 slots, a rotation at far positions, weights spread and peaked."""
    for boost in (1.0, 6.0):
        c = Case(km.F16, 1, 5, 128, 128, [40000], 5, mode=2, rot=128, seed=3)
        c.q *= np.float32(boost)
        for chunk in (0, 1024):
            c.check(c.run(chunk=chunk), chunk=chunk or 4096)


@pytest.mark.parametrize("kind", KINDS)
def test_sizes_of_q(kind):
    """Queries of any magnitude keep fp32 accuracy (scores stay moderate:
    the scale goes the other way)."""
    for power in (-80, -20, 20, 80):
        c = Case(KINDS[kind], 1, 2, 64, 32, [100], 4)
        c.q *= np.float32(2.0 ** power)
        c.scale *= 2.0 ** -power
        c.check(c.run())


@pytest.mark.parametrize("low,high", [(-6, 6), (-60, -60), (100, 100), (-75, -70), (0, 12)])
def test_sizes_of_int8_values(low, high):
    """Value scales of any size, and different ones in the slots of a row."""
    c = Case(km.I8, 2, 3, 64, 32, [700, 45], 4)
    rng = np.random.default_rng(8)
    k, v = rows(rng, 2, 700, 2, 64)
    v *= (2.0 ** rng.integers(low, high + 1, (2, 700, 2, 1))).astype(np.float32)
    nk, nv = rows(rng, 2, 4, 2, 64)
    nv *= np.float32(2.0 ** low)
    c.kv.lens.zero_()
    c.kv.append(1, dev(k), dev(v), n_new=ints(c.lens))
    c.kv.lens.copy_(ints(c.lens))
    c.kv.append(1, dev(nk), dev(nv))
    for b, n in enumerate(c.lens):
        c.k[b, :n], c.v[b, :n] = km.stored(k[b, :n], km.I8), km.stored(v[b, :n], km.I8)
        c.k[b, n:n + 4], c.v[b, n:n + 4] = km.stored(nk[b], km.I8), km.stored(nv[b], km.I8)
    for chunk in (0, 128, 640):
        c.check(c.run(chunk=chunk), chunk=chunk or 4096)


# ------------------------------------------------- streams, graphs, wrapper
def cycle(kv, plan, M, q, k, v, out, acc, tree, rope):
    kv.reserve(M)
    for layer in range(kv.layers):
        kv.append(layer, k, v, tree=tree, rope=rope)
        plan.run(layer, q, out[layer], tree=tree, rope=rope)
    kv.commit(M, acc)


def test_a_cycle_replayed():
    """Reserve, append, attention and commit captured once and replayed, with
    eager work between the replays, equal the eager calls; a second graph
    with a plan of its own runs between them."""
    t = torch()
    rng = np.random.default_rng(8)
    B, M, H, G, D = 2, 4, 2, 3, 64
    kv, ref = (sv.KvCache(km.F16, 2, H, D, 32, 64, B, 12) for _ in "ab")
    for c in (kv, ref):
        c.data.zero_()
    rope = sv.Rope(2, D, sv.rope_table(12 * 32, D))
    tree = ints([[1, 3, 7, 11]] * B)
    k, v, q = (t.empty((B, M, n, D), device="cuda") for n in (H, H, H * G))
    acc = ints([2, 0])
    out = [t.zeros((B, M, H * G, D), device="cuda") for _ in range(2)]
    plan, eager, other = (c.attention(H * G, B, M, chunk=128) for c in (kv, ref, kv))
    side = t.cuda.Stream()
    spare = t.zeros_like(out[0])
    with t.cuda.stream(side):
        eager.run(0, q, spare)
    side.synchronize()
    graph, second = t.cuda.CUDAGraph(), t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        cycle(kv, plan, M, q, k, v, out, acc, tree, rope)
    with t.cuda.graph(second):
        other.run(1, q, spare, tree=tree, rope=rope)
    want = [t.zeros_like(out[0]) for _ in range(2)]
    for i in range(12):
        for x in (k, v, q):
            x.copy_(dev(rng.standard_normal(tuple(x.shape)).astype(np.float32)))
        acc.copy_(ints([int(rng.integers(-1, M)), int(rng.integers(0, M))]))
        graph.replay()
        second.replay()
        cycle(ref, eager, M, q, k, v, want, acc, tree, rope)
        for a, b in zip(out, want):
            assert np.array_equal(host(a), host(b)), i
        for n in ("table", "lens", "refs", "ctl"):
            assert np.array_equal(host(getattr(kv, n)), host(getattr(ref, n))), (i, n)
        kv.read(1, k)
        assert np.array_equal(host(kv.data), host(ref.data)), i
    assert kv.status() == 0


def test_calls_on_a_stream():
    """Calls go to the current stream, or the one given."""
    t = torch()
    c = Case(km.F16, 2, 2, 64, 32, [300, 20], 4)
    want = c.run(chunk=128)
    q, out = dev(c.q), t.empty((2, 4, 4, 64), device="cuda")
    plan = c.kv.attention(4, 2, 4, chunk=128)
    side = t.cuda.Stream()
    t.cuda.synchronize()
    with t.cuda.stream(side):
        plan.run(1, q, out)
    side.synchronize()
    assert np.array_equal(out.cpu().numpy(), want)
    out.zero_()
    t.cuda.synchronize()
    plan.run(1, q, out, stream=side)
    side.synchronize()
    assert np.array_equal(out.cpu().numpy(), want)


def test_the_wrapper_refuses():
    t = torch()
    kv = sv.KvCache(km.F16, 1, 2, 64, 32, 8, 2, 4)
    kv.reserve(4)
    good = t.zeros((2, 4, 2, 64), device="cuda")
    for bad in (good.cpu(), good.half(), good.transpose(0, 1), t.zeros((2, 4, 2, 32), device="cuda"),
                t.zeros((2, 4, 2, 128), device="cuda")[..., ::2]):
        with pytest.raises(sv.SpecVerifyError):
            kv.append(0, good, bad)
        with pytest.raises(sv.SpecVerifyError):
            kv.read(0, good, bad)
    plan = kv.attention(4, 2, 4)
    q = t.zeros((2, 4, 4, 64), device="cuda")
    for args in ((0, q[:1]), (0, q, good), (0, q.double(), q), (1, q, q), (0, q, None)):
        with pytest.raises(sv.SpecVerifyError):
            plan.run(*args)
    with pytest.raises(sv.SpecVerifyError):
        plan.run(0, q, q, n_new=t.zeros(2, dtype=t.int64, device="cuda"))
    with pytest.raises(sv.SpecVerifyError):
        plan.run(0, q, q, seq=t.zeros(3, dtype=t.int32, device="cuda"))
    with pytest.raises(sv.SpecVerifyError):
        kv.attention(5, 2, 4).run(0, q, q)
    with pytest.raises(sv.SpecVerifyError):
        kv.commit(4, ints([1]))
    with pytest.raises(sv.SpecVerifyError):
        kv.fork(ints([0]), ints([0, 1]))
    with pytest.raises(sv.SpecVerifyError):
        sv.KvCache(km.F16, 1, 2, 100, 32, 8, 2, 4)
    with pytest.raises(sv.SpecVerifyError):
        sv.KvCache(km.F16, 1, 2, 64, 32, 8, 2, 4, buffers={n: getattr(kv, n if n != "len" else "lens")[:1]
                                                            for n in ("data", "table", "len", "refs", "free_ids", "ctl")})
    with pytest.raises(sv.SpecVerifyError):
        sv.Rope(2, 64, t.zeros((128, 16, 2), device="cuda"))
    assert kv.status() == 0
