"""Attention of a batch whose sequences share their first slots: every row's
bits are those of the attention that does not share, and both agree with the
definition in 64 bits."""

import numpy as np
import pytest

import kv_model as km
import speculative_decoding_verification_amd as sv
from gpu_util import dev, host, torch

pytestmark = pytest.mark.gpu

KINDS = {"f16": km.F16, "bf16": km.BF16, "i8": km.I8}


def ints(x):
    return dev(np.asarray(x, np.int32))


class Forks:
    """Sequences that continue one prompt, made by the page calls: a prompt of
    `prompt` rows forked B - 1 times, each then with `own[b]` rows of its own
    and M new ones."""

    def __init__(self, kind, heads, group, dim, page, prompt, own, M, n_new=None, tree=None, mode=0, rot=0, seed=0):
        self.rng = rng = np.random.default_rng(seed)
        B = self.B = len(own)
        self.heads, self.group, self.dim, self.M = heads, group, dim, M
        self.shared = prompt // page * page
        self.n_new = [M] * B if n_new is None else n_new
        self.n_arg = None if n_new is None else ints(n_new)
        self.tree = None if tree is None else ints(tree)
        self.masks = tree
        width = -(-(prompt + max(own) + M) // page)
        self.kv = kv = sv.KvCache(kind, 1, heads, dim, page, (B + 1) * width + 2, B + 2, width)
        kv.data.fill_(0xFF)
        self.seq = ints(rng.permutation(B + 2)[:B])
        self.rope = sv.Rope(mode, rot, sv.rope_table(width * page, rot)) if mode else None
        rows = lambda n, m: [(rng.standard_normal((n, m, heads, dim)) * 2).astype(np.float32) for _ in "kv"]  # noqa: E731
        first = self.seq[:1].contiguous()
        k, v = rows(1, max(prompt, 1))
        if prompt:
            kv.reserve(prompt, seq=first)
            kv.append(0, dev(k), dev(v), seq=first)
            kv.commit(prompt, ints([prompt - 1]), seq=first)
        if B > 1:
            kv.fork(first.expand(B - 1).contiguous(), self.seq[1:].contiguous())
        self.own = own
        if max(own):
            k, v = rows(B, max(own))
            kv.reserve(max(own), seq=self.seq, n_new=ints(own))
            kv.append(0, dev(k), dev(v), seq=self.seq, n_new=ints(own))
            kv.commit(max(own), ints(np.asarray(own) - 1), seq=self.seq, n_new=ints(own))
        kv.reserve(M, seq=self.seq, n_new=self.n_arg)
        k, v = rows(B, M)
        kv.append(0, dev(k), dev(v), seq=self.seq, n_new=self.n_arg, tree=self.tree, rope=self.rope)
        assert kv.status() == 0
        self.lens = [prompt + n for n in own]
        assert host(kv.lens)[host(self.seq)].tolist() == self.lens
        self.q = dev((rng.standard_normal((B, M, heads * group, dim)) * 1.5).astype(np.float32))

    def plan(self, shared, chunk=0, **kw):
        return self.kv.attention(self.heads * self.group, self.B, self.M, chunk=chunk, shared=shared, **kw)

    def run(self, plan, q=None, ep=None, seq=None):
        out = torch().full((self.B, self.M, self.heads * self.group, self.dim), 77.0, device="cuda")
        plan.run(0, self.q if q is None else q, out, seq=self.seq if seq is None else seq, n_new=self.n_arg, tree=self.tree,
                 rope=self.rope, ep=ep)
        return host(out)

    def check(self, got, chunk):
        """Every sequence against the definition, its slots read back."""
        kv, t = self.kv, torch()
        for b in range(self.B):
            n, new = self.lens[b], self.n_new[b]
            assert (got[b, new:] == 77).all()
            if not new:
                continue
            k = t.empty((1, n + new, self.heads, self.dim), device="cuda")
            v = t.empty_like(k)
            kv.read(0, k, v, seq=self.seq[b:b + 1].contiguous(), start=ints([0]))
            masks = [(2 << m) - 1 for m in range(self.M)] if self.masks is None else self.masks[b]
            rope = (0, 0, None) if self.rope is None else (self.rope.c.mode, self.rope.c.rot, host(self.rope.table))
            q = np.stack([km.rotated(host(self.q)[b, m], n + km.depth(masks, m), *rope) for m in range(self.M)])
            want, mag, amp = km.attention(q, host(k)[0], host(v)[0], n, new, self.dim ** -0.5, masks=masks)
            err = np.abs(got[b, :new] - want)
            assert (err <= km.attention_bound(mag, amp, self.dim, n + new, chunk)).all(), (b, err.max())
            assert np.linalg.norm(err) <= km.norm_bound(amp, self.dim) * np.linalg.norm(want), b


TREE = np.array([[1, 3, 5, 11, 21, 0, 65, 128 + 21], [1, 2, 4, 8, 16, 32, 64, 255], [1, 3, 7, 15, 31, 63, 127, 255]], np.int32)

SHAPES = [  # kind, heads, group, dim, page, prompt, own, M
    ("f16", 2, 5, 128, 64, 1000, [60, 3, 17, 0], 1), ("bf16", 2, 5, 128, 64, 700, [200, 1, 90], 5),
    ("i8", 3, 2, 96, 128, 900, [10] * 9, 3), ("f16", 1, 1, 32, 32, 513, [0] * 70, 1), ("bf16", 1, 1, 64, 32, 300, [5] * 40, 2),
    ("i8", 2, 4, 64, 256, 1100, [700, 5], 16), ("f16", 1, 8, 160, 64, 400, [33, 34, 35], 4), ("bf16", 1, 3, 256, 64, 290, [9, 0], 6),
    ("i8", 1, 64, 128, 64, 260, [1, 2], 2), ("f16", 8, 1, 64, 64, 640, [0, 64, 128], 1), ("i8", 1, 5, 224, 32, 384, [2, 3], 7),
    ("bf16", 4, 2, 192, 128, 256, [0, 0, 0], 1), ("f16", 2, 7, 96, 32, 2000, [40, 80, 120, 160, 200], 8),
    ("bf16", 3, 4, 32, 64, 777, [12, 300], 9)]


@pytest.mark.parametrize("kind,heads,group,dim,page,prompt,own,M", SHAPES)
def test_rows_equal_those_without_sharing(kind, heads, group, dim, page, prompt, own, M):
    f = Forks(KINDS[kind], heads, group, dim, page, prompt, own, M, mode=2, rot=dim)
    for chunk in (128, 256, 384):
        want = f.run(f.plan(0, chunk))
        for shared in sorted({f.shared, max(0, f.shared - page), 130 if f.shared > 130 else 0}):
            assert np.array_equal(f.run(f.plan(shared, chunk)), want), (chunk, shared)
    f.check(want, 384)
    f.check(f.run(f.plan(f.shared)), 1 << 14)
    assert f.kv.status() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("mode,rot", [(0, 0), (1, 64), (2, 32), (2, 6), (1, 10)])
@pytest.mark.parametrize("group,M", [(1, 1), (4, 8), (3, 2)])
def test_rotations_rows_and_trees(kind, mode, rot, group, M):
    """Ragged numbers of new rows (some without any), draft trees, rotations
    with and without whole quads of pairs."""
    tree = TREE[[0, 1, 2, 0, 1, 2]][:, :M] & ((1 << M) - 1)
    for use in (None, tree):
        f = Forks(KINDS[kind], 2, group, 64, 32, 420, [7, 40, 1, 0, 90, 3], M, n_new=[M, 1, 0, M, max(1, M - 1), M], tree=use,
                  mode=mode, rot=rot, seed=M)
        want = f.run(f.plan(0, 128))
        assert np.array_equal(f.run(f.plan(f.shared, 128)), want)
        f.check(want, 128)


def test_a_long_prefix_and_many_sequences():
    """A batch above one wave's lanes, and chunks of the rule's choice."""
    f = Forks(km.F16, 2, 4, 64, 64, 5000, [(7 * b) % 150 for b in range(100)], 2, mode=2, rot=64)
    plan = f.plan(f.shared)
    got = f.run(plan)
    f.check(got, 1 << 14)
    for chunk in (512, 2048):
        assert np.array_equal(f.run(f.plan(f.shared, chunk)), f.run(f.plan(0, chunk)))


def test_the_requantised_output():
    f = Forks(km.F16, 2, 4, 64, 64, 600, [50, 2, 9], 3)
    rows, K = 9, 8 * 64
    t = torch()
    new = lambda n, dt: t.zeros((rows, n), dtype=dt, device="cuda")  # noqa: E731
    got = dict(q=new(K, t.int8), d=new(K // 32, t.float32), s16=new(K // 16, t.int32), sumsq=new(K // 32, t.float32))
    g = dev((1 + 0.1 * f.rng.standard_normal(K)).astype(np.float32))
    out = f.run(f.plan(f.shared, 128), ep=sv.epilogue(sv.SV_EP_QUANT, got["q"], got["d"], got["s16"], got["sumsq"], gamma=g))
    want = dict(q=new(K, t.int8), d=new(K // 32, t.float32), s16=new(K // 16, t.int32), sumsq=new(K // 32, t.float32))
    sv.quantize_act_q8(dev(out).view(rows, K), want["q"], want["d"], want["s16"], gamma=g, sumsq=want["sumsq"])
    for n in got:
        assert t.equal(got[n], want[n]), n


def test_sequences_that_do_not_share_are_refused():
    """Another page, fewer slots, an index out of range: NaN and a status for
    that sequence, the others as ever; what is not shared may differ."""
    f = Forks(km.BF16, 2, 3, 64, 64, 600, [50, 2, 9, 30], 2)
    plan, want = f.plan(f.shared, 128), f.run(f.plan(0, 128))
    kv, seq = f.kv, host(f.seq)
    kept = [x.clone() for x in kv.bookkeeping()]

    def restore():
        for x, y in zip(kv.bookkeeping(), kept):
            x.copy_(y)

    def expect(bad, bits):
        got = f.run(plan)
        for b in range(4):
            if b in bad:
                assert np.isnan(got[b]).all(), b
            else:
                assert np.array_equal(got[b], want[b]), b
        assert kv.status() == bits
        restore()

    expect([], 0)
    kv.table[int(seq[2]), 3] = kv.table[int(seq[2]), 5].clone()   # another page inside the shared chunks
    expect([2], sv.SV_KV_NOT_SHARED)
    kv.table[int(seq[1]), 0] = -1
    expect([1], sv.SV_KV_NOT_SHARED)
    kv.table[int(seq[0]), 4] = -1                                 # the first: then nobody shares
    expect([0, 1, 2, 3], sv.SV_KV_NOT_SHARED)
    kv.lens[int(seq[3])] = 100
    expect([3], sv.SV_KV_NOT_SHARED)
    kv.lens[int(seq[3])] = 0
    expect([3], sv.SV_KV_NOT_SHARED)
    # 576 slots in whole chunks of 128 are 512: what lies past them is each one's own
    kv.table[int(seq[3]), 8] = kv.table[int(seq[3]), 9].clone()
    # (some slots of the page that it now holds there were never written: NaN, as without sharing)
    got = f.run(plan)
    assert kv.status() == 0 and np.array_equal(got, f.run(f.plan(0, 128)), equal_nan=True)
    assert np.array_equal(got[:3], want[:3])
    restore()
    # a sequence out of range has no rows; out of range as the first, nobody shares
    other = f.seq.clone()
    other[2] = 99
    got = f.run(plan, seq=other)
    assert (got[2] == 77).all() and np.array_equal(got[[0, 1, 3]], want[[0, 1, 3]]) and kv.status() == 0
    other = f.seq.clone()
    other[0] = -1
    got = f.run(plan, seq=other)
    assert (got[0] == 77).all() and np.isnan(got[1:]).all() and kv.status() == sv.SV_KV_NOT_SHARED
    # the same sequence twice
    other = f.seq.clone()
    other[3] = other[1]
    got = f.run(plan, seq=other)
    assert np.array_equal(got[:3], want[:3]) and kv.status() == 0


def test_rows_with_nothing_new_lead():
    """The first sequence lends its pages also where it has no rows."""
    f = Forks(km.I8, 1, 2, 64, 32, 300, [5, 6, 7], 4, n_new=[0, 4, 2])
    assert np.array_equal(f.run(f.plan(f.shared, 128)), f.run(f.plan(0, 128)))


def test_queries_that_are_not_finite_stay_in_their_rows():
    f = Forks(km.F16, 1, 2, 64, 64, 520, [5, 6, 7, 8], 2)
    want = f.run(f.plan(f.shared, 128))
    q = f.q.clone()
    q[1, 1, 0, 5], q[2, 0, 1, 7] = float("nan"), float("inf")
    got = f.run(f.plan(f.shared, 128), q=q)
    assert np.array_equal(got, f.run(f.plan(0, 128), q=q), equal_nan=True)
    assert np.isnan(got[1, 1, 0]).all() and np.isnan(got[2, 0, 1]).any()
    ok = np.ones(got.shape[:3], bool)
    ok[1, 1, 0] = ok[2, 0, 1] = False
    assert np.array_equal(got[ok], want[ok])


@pytest.mark.parametrize("kind", KINDS)
def test_large_scores_and_odd_values(kind):
    """Scores past 2^24, and values that are not finite in a shared slot."""
    f = Forks(KINDS[kind], 1, 2, 64, 64, 520, [5, 6, 7], 2)
    f.q.mul_(1e7)
    assert np.array_equal(f.run(f.plan(f.shared, 128)), f.run(f.plan(0, 128)))
    k = torch().zeros((1, 1, 1, 64), device="cuda")
    v = k.clone()
    v[..., 3] = float("inf")
    one = f.seq[:1].contiguous()
    n = f.kv.lens[int(f.seq[0])].clone()
    f.kv.lens[int(f.seq[0])] = 200
    f.kv.append(0, k, v, seq=one)
    f.kv.lens[int(f.seq[0])] = n
    f.q.mul_(1e-8)
    got = f.run(f.plan(f.shared, 128))
    assert np.array_equal(got, f.run(f.plan(0, 128)), equal_nan=True)
    assert not np.isfinite(got[:, :, :, 3]).any()


def test_longer_than_max_len():
    f = Forks(km.F16, 1, 2, 64, 64, 520, [5, 60, 7], 2)
    plan = f.plan(f.shared, 128, max_len=540)
    got = f.run(plan)
    assert np.isnan(got[1]).all() and np.array_equal(got[[0, 2]], f.run(f.plan(0, 128))[[0, 2]])
    assert f.kv.status() == sv.SV_KV_OVER_MAX
    plan = f.plan(f.shared, 128, max_len=130)      # shorter than the shared slots
    assert np.isnan(f.run(plan)).all()
    assert f.kv.status() & sv.SV_KV_OVER_MAX


def test_a_cycle_replayed_with_eager_work_between():
    """Two captured rounds with plans of their own, replayed in turn with
    eager calls between them."""
    t = torch()
    f = Forks(km.F16, 2, 4, 64, 64, 1000, [50, 2, 9], 3, mode=2, rot=64)
    plans = [f.plan(f.shared, c) for c in (128, 256)]
    qs = [dev((f.rng.standard_normal(f.q.shape) * 1.5).astype(np.float32)) for _ in range(3)]
    want = [[f.run(f.plan(0, c), q=q) for q in qs] for c in (128, 256)]
    q, out = qs[0].clone(), [t.zeros_like(f.q) for _ in plans]
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        for p, o in zip(plans, out):
            p.run(0, q, o, seq=f.seq, rope=f.rope)
    t.cuda.current_stream().wait_stream(side)
    t.cuda.synchronize()
    graphs = []
    for p, o in zip(plans, out):
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            p.run(0, q, o, seq=f.seq, rope=f.rope)
        graphs.append(g)
    for i in (1, 0, 2, 1):
        q.copy_(qs[i])
        for o in out:
            o.zero_()
        for g in graphs:
            g.replay()
        f.run(f.plan(f.shared))
        for w, o in zip(want, out):
            assert np.array_equal(host(o), w[i])


def test_a_round_of_continuations():
    """The operators together: one prompt forked, a round of every sequence
    with shared attention, the residual's norm, a head, sampling, commit; and
    the same sequences run one by one give the same tokens."""
    import synth
    from gpu_util import upload_weight
    t = torch()
    heads, group, dim, page, B = 2, 4, 32, 32, 5
    H, V = heads * group * dim, 1000
    f = Forks(km.F16, heads, group, dim, page, 300, [0] * B, 1, mode=2, rot=dim, seed=3)
    head, keep = upload_weight(sv.SV_Q8_0, synth.gguf_weights(sv.SV_Q8_0, V, H, 1, "H"), H)
    x = dev(f.rng.standard_normal((B, H)).astype(np.float32))
    gamma = dev((1 + 0.1 * f.rng.standard_normal(H)).astype(np.float32))
    params, u = sv.sampling_params(40.0, 50, 0.95, 0.0), dev(f.rng.random(B))

    def round_of(rows, shared):
        n = len(rows)
        plan = f.kv.attention(heads * group, n, 1, chunk=128, shared=shared)
        o = t.zeros((n, 1, heads * group, dim), device="cuda")
        plan.run(0, f.q[rows].contiguous(), o, seq=f.seq[rows].contiguous(), rope=f.rope)
        new = lambda k, dt: t.zeros((n, k), dtype=dt, device="cuda")  # noqa: E731
        s, q, d, s16, ss = new(H, t.float32), new(H, t.int8), new(H // 32, t.float32), new(H // 16, t.int32), new(H // 32, t.float32)
        sv.add_norm_q8(x[rows].contiguous(), o.view(n, H), gamma=gamma, fold=True, sum=s, q=q, d=d, s16=s16, sumsq=ss)
        logits, tok = new(V, t.float32), t.zeros(n, dtype=t.int32, device="cuda")
        sv.head_logits(head, sv.act(n, H, q, d, s16, ss, H // 32), logits)
        sv.sample(logits, params, u[rows].contiguous(), tok, sv.sample_workspace(n, V))
        return host(tok).tolist(), host(s)

    together, s = round_of(list(range(B)), f.shared)
    assert all(0 <= x < V for x in together) and len(set(together)) > 1
    for b in range(B):
        tok, sb = round_of([b], 0)
        assert tok == [together[b]] and np.array_equal(sb[0], s[b])
    f.kv.commit(1, t.zeros(B, dtype=t.int32, device="cuda"), seq=f.seq)
    assert host(f.kv.lens)[host(f.seq)].tolist() == [301] * B and f.kv.status() == 0
