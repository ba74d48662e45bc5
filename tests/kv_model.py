"""A plain model of the key-value cache, written from its description: page
bookkeeping one sequence and one entry at a time, rows as numbers, attention
in 64 bits.  It shares no code with the GPU library."""

from __future__ import annotations

import math

import numpy as np

F16, BF16, I8 = 1, 30, 24
NO_PAGES, TOO_LONG, BAD_FORK, NO_SLOT, BAD_COMMIT, OVER_MAX = 1, 2, 4, 8, 16, 32


def bf16(x):
    """fp32 rounded to bf16 (nearest, ties to even), as fp32."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32)
    nan = np.isnan(x)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(nan, np.float32(np.nan), r)


def stored(x, kind):
    """What a row x[..., dim] of fp32 is in a cache, as fp32."""
    x = np.asarray(x, np.float32)
    if kind == F16:
        with np.errstate(over="ignore"):
            return x.astype(np.float16).astype(np.float32)
    if kind == BF16:
        return bf16(x)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        fine = np.isfinite(x).all(-1, keepdims=True)
        d = (np.abs(x).max(-1, keepdims=True) / np.float32(127)).astype(np.float32)
        d = np.where(d >= np.float32(2.0 ** -126), d, np.float32(0))
        t = (x * np.where(d > 0, np.float32(1) / d, np.float32(0))).astype(np.float32)
        q = np.clip(np.sign(t) * np.floor(np.abs(t).astype(np.float64) + 0.5), -127, 127).astype(np.float32)
        return np.where(fine, (q * d).astype(np.float32), np.float32(np.nan))


def rotated(x, pos, mode, rot, table):
    """x [heads, dim] at a position: products and sums in fp32."""
    if mode == 0:
        return x
    y = x.astype(np.float32).copy()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if mode == 1 else (i, i + rot // 2)
        c, s = table[pos, i]
        y[:, a] = x[:, a] * c - x[:, b] * s
        y[:, b] = x[:, b] * c + x[:, a] * s
    return y


def depth(masks, m):
    return bin(int(masks[m]) & ((1 << m) - 1)).count("1")


class Model:
    """The cache of one layer (the bookkeeping is the same for all)."""

    def __init__(self, kind, heads, dim, page, n_pages, seqs, width):
        self.kind, self.heads, self.dim, self.page = kind, heads, dim, page
        self.n_pages, self.seqs, self.width = n_pages, seqs, width
        self.table = np.full((seqs, width), -1, np.int32)
        self.len = np.zeros(seqs, np.int32)
        self.refs = np.zeros(n_pages, np.int32)
        self.free = list(range(n_pages - 1, -1, -1))
        self.status = 0
        self.k = np.zeros((n_pages, page, heads, dim), np.float32)
        self.v = np.zeros((n_pages, page, heads, dim), np.float32)

    def first(self, seq):
        seen = set()
        for b, s in enumerate(seq):
            if 0 <= s < self.seqs and s not in seen:
                seen.add(s)
                yield b, s

    def reserve(self, n, seq, n_new=None):
        want = []
        for b, s in self.first(seq):
            rows = n if n_new is None else min(max(int(n_new[b]), 0), n)
            lo, hi = -(-int(self.len[s]) // self.page), -(-(int(self.len[s]) + rows) // self.page)
            if hi > self.width:
                self.status |= TOO_LONG
                return
            want += [(s, e) for e in range(lo, hi) if self.table[s, e] < 0]
        if len(want) > len(self.free):
            self.status |= NO_PAGES
            return
        for s, e in want:
            p = self.free.pop()
            self.table[s, e], self.refs[p] = p, 1

    def place(self, s, slot):
        if slot < 0 or slot >= self.width * self.page:
            return None
        p = self.table[s, slot // self.page]
        return (p, slot % self.page) if 0 <= p < self.n_pages else None

    def append(self, k, v, seq, n_new=None, tree=None, rope=(0, 0, None)):
        B, M = k.shape[:2]
        for b, s in self.first(seq):
            rows = M if n_new is None else min(max(int(n_new[b]), 0), M)
            masks = [(2 << m) - 1 for m in range(M)] if tree is None else tree[b]
            for m in range(rows):
                slot = int(self.len[s]) + m
                at = self.place(s, slot)
                if at is None:
                    self.status |= NO_SLOT
                    continue
                self.k[at] = stored(rotated(k[b, m], int(self.len[s]) + depth(masks, m), *rope), self.kind)
                self.v[at] = stored(v[b, m], self.kind)

    def read(self, s, start, n):
        k = np.zeros((n, self.heads, self.dim), np.float32)
        v = np.zeros_like(k)
        for i in range(n):
            at = self.place(s, start + i)
            if at is not None:
                k[i], v[i] = self.k[at], self.v[at]
        return k, v

    def drop(self, entries):
        """entries (s, e) in order: a page goes on the free list at the last
        entry naming it once nobody holds it."""
        last = {}
        for i, (s, e) in enumerate(entries):
            p = self.table[s, e]
            self.refs[p] -= 1
            last[p] = i
        for i, (s, e) in enumerate(entries):
            p = self.table[s, e]
            if self.refs[p] == 0 and last[p] == i:
                self.free.append(int(p))
        for s, e in entries:
            self.table[s, e] = -1

    def commit(self, M, accepted, seq, n_new=None, path=None):
        gone = []
        for b, s in self.first(seq):
            rows = M if n_new is None else min(max(int(n_new[b]), 0), M)
            kept = int(accepted[b]) + 1 if accepted[b] >= 0 else 0
            n = int(self.len[s])
            p = [int(x) for x in path[b][:kept]] if path is not None else list(range(kept))
            ok = kept <= rows and all(0 <= r < rows for r in p) and all(x < y for x, y in zip(p, p[1:]))
            if not ok or (kept and self.place(s, n + kept - 1) is None):
                self.status |= BAD_COMMIT
                continue
            for i, r in enumerate(p):
                a, z = self.place(s, n + r), self.place(s, n + i)
                if a is not None and z is not None and a != z:
                    self.k[z], self.v[z] = self.k[a], self.v[a]
            self.len[s] = n + kept
            gone += [(s, e) for e in range(-(-(n + kept) // self.page), self.width) if self.table[s, e] >= 0]
        self.drop(gone)

    def fork(self, src, dst):
        bad = any(not (0 <= s < self.seqs and 0 <= d < self.seqs) for s, d in zip(src, dst)) or \
            len(set(dst)) < len(dst) or set(dst) & set(src)
        bad = bad or any(self.len[d] or self.table[d, 0] >= 0 for d in dst)
        if bad:
            self.status |= BAD_FORK
            return
        part = [self.len[s] % self.page != 0 and self.table[s, self.len[s] // self.page] >= 0 for s in src]
        if sum(part) > len(self.free):
            self.status |= NO_PAGES
            return
        for s, d, copy in zip(src, dst, part):
            full = self.len[s] // self.page
            self.table[d, :full] = self.table[s, :full]
            for p in self.table[s, :full]:
                self.refs[p] += 1
            if copy:
                p, old = self.free.pop(), self.table[s, full]
                self.table[d, full], self.refs[p] = p, 1
                used = self.len[s] % self.page
                self.k[p, :used], self.v[p, :used] = self.k[old, :used], self.v[old, :used]
            self.len[d] = self.len[s]

    def release(self, ids):
        gone = []
        for _, s in self.first(ids):
            gone += [(s, e) for e in range(self.width) if self.table[s, e] >= 0]
            self.len[s] = 0
        self.drop(gone)

    def compact(self):
        live = self.n_pages - len(self.free)
        holes = [p for p in range(live) if self.refs[p] == 0]
        moves = [p for p in range(live, self.n_pages) if self.refs[p] > 0]
        for old, new in zip(moves, holes):
            self.k[new], self.v[new] = self.k[old], self.v[old]
            self.refs[new], self.refs[old] = self.refs[old], 0
            self.table[self.table == old] = new
        self.free = list(range(self.n_pages - 1, live - 1, -1))


def attention(q, k, v, length, n, scale, held=None, masks=None, window=0, sinks=0):
    """One sequence in 64 bits.  q [M, q_heads, dim]; k, v [slots, heads,
    dim] of the slots 0..length+n-1; held [slots]: the slot has a page.
    Returns out [n, q_heads, dim], the weighted sum of |v| and the largest
    sum of |q k| * scale of each row (what its rounding errors scale with)."""
    Hq, H, D = q.shape[1], k.shape[1], q.shape[2]
    S = length + n
    masks = [(2 << m) - 1 for m in range(n)] if masks is None else [int(x) for x in masks[:n]]
    pos = np.arange(S)
    for m in range(n):
        pos[length + m] = length + depth(masks, m)
    out = np.zeros((n, Hq, D))
    mag = np.zeros((n, Hq, D))
    amp = np.zeros((n, Hq))
    for m in range(n):
        vis = np.ones(S, bool)
        for t in range(n):
            vis[length + t] = masks[m] >> t & 1
        mine = length + depth(masks, m)
        if window:
            vis &= (mine - pos < window) | (pos < sinks)
        if held is not None:
            vis &= held[:S]
        if not vis.any():
            continue
        idx = np.nonzero(vis)[0]
        for h in range(Hq):
            kk, vv = k[idx, h // (Hq // H)].astype(np.float64), v[idx, h // (Hq // H)].astype(np.float64)
            qq = q[m, h].astype(np.float64)
            with np.errstate(invalid="ignore", over="ignore"):
                s = kk @ qq * scale
                w = np.exp(s - s.max())
                w /= w.sum()
                out[m, h] = w @ vv
                mag[m, h] = w @ np.abs(vv)
                amp[m, h] = (np.abs(kk) @ np.abs(qq)).max() * scale
    return out, mag, amp


def attention_bound(mag, amp, dim, slots, chunk):
    """Largest rounding error of the fp32 attention, per output.

    Half a step of fp32 is u = 2^-24.  A score is a sum of at most 3 dim
    products (three parts of q), each addition off by u of the running
    magnitude; q has been scaled (u) and split (the rest after two fp16 or
    three bf16 parts is at most 2^-22 = 4 u of the element); int8 scores are
    scaled twice more, the exponent is rounded and 2^x is good to 2 u: a
    weight is off by at most (3 dim + 16) u amp + 4 u relative, in the sums
    above and below the line alike.  An output is a sum of at most 96
    products (three parts, 32 slots) for each block of a wave's share of a
    chunk (half of one at most, in blocks of 32), then of up to 8 waves and
    the chunks; weights are split as q is, and what is left of one is at most
    2^-39 of the row's largest weight (int8: with its scale), which is below
    these sums' roundings unless weights of 2^-15 make up an output.
    """
    u = 2.0 ** -24
    weight = ((3 * dim + 16) * amp[..., None] + 4) * u
    adds = (96 * -(-chunk // 64) + 8 + -(-slots // chunk) + 16) * u
    return (2 * weight + 2 * adds) * mag + 1e-37


def norm_bound(amp, dim):
    """The same errors as independent roundings: the 2-norm of a difference
    over the 2-norm of the result, with four times its expected size."""
    return 4 * math.sqrt(3 * dim + 16 + 96) * 2.0 ** -24 * max(1.0, float(amp.max()) / math.sqrt(dim))
