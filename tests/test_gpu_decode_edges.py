"""Sampling, the residual's norm and attention over shared slots where their
ways of working change: lists that overflow, rows under way at once, lengths
about a border of the kernels' pieces, offsets past 32 bits, calls that run
side by side."""

import numpy as np
import pytest

import kv_model as km
import speculative_decoding_verification_amd as sv
from gpu_util import dev, host, torch
from test_gpu_decode import check_sample, draw_settings, logits_of, norm_buffers, run_sample
from test_gpu_shared import Forks

pytestmark = pytest.mark.gpu

# top-k alone, top-p alone, min-p alone, and together: within a list, past it,
# and past it by count and mass at once
SETTINGS = [(1.0, 40, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (1.0, 0, 1.0, 0.1), (0.7, 40, 0.9, 0.05), (1.0, 0, 0.05, 0.0),
            (1.0, 3000, 1.0, 0.0), (1.0, 9000, 0.7, 0.0), (2.0, 9000, 1.0, 0.3), (1.0, 0, 0.9, 0.3), (1.0, 0, 1.0, 0.0),
            (1.0, 9000, 0.3, 0.6), (0.0, 0, 1.0, 0.0)]


@pytest.mark.parametrize("V", [2559, 2560, 2561, 8191, 8192, 8193, 12287, 12288, 16387, 32767, 32768, 65537])
@pytest.mark.parametrize("kind", ["peaked", "flat", "ties"])
def test_lengths_about_the_pieces(V, kind):
    rng = np.random.default_rng(V)
    z, u = logits_of(rng, len(SETTINGS), V, kind), rng.random(len(SETTINGS))
    check_sample(z, SETTINGS, u, run_sample(z, SETTINGS, u))


def shapes_of(rng, rows, V, kind):
    z = rng.standard_normal((rows, V))
    if kind == "one chunk":          # the large ones side by side, more than a chunk's list holds
        at = int(rng.integers(0, V - 6000))
        z[:, at:at + 6000] += 12
    elif kind == "even":             # by mass and by count a border among very many
        z = rng.random((rows, V))
    elif kind == "two values":       # equal elements, more than a list holds
        z = (rng.random((rows, V)) < 0.6) * 1.0
    elif kind == "a step":           # a flat floor under a few large ones
        z *= 1e-3
        z[:, rng.integers(0, V, 30)] += 9
    elif kind == "one far above":    # nothing else has a weight that counts
        z[:, V // 3] += 90
    elif kind == "a few":            # fewer are finite than the settings ask for
        z[rng.random((rows, V)) < 0.98] = -np.inf
    elif kind == "close":            # neighbours a rounding apart
        z = 1 + rng.integers(0, 4000, (rows, V)) * 2.0 ** -23
    elif kind == "far":              # the sample's largest lies far below the row's
        z[:, :] = -1e4 + z
        z[:, V // 2 + 77] = 3e4
    return z.astype(np.float32)


@pytest.mark.parametrize("V", [20011, 151936])
@pytest.mark.parametrize("kind", ["one chunk", "even", "two values", "a step", "one far above", "a few", "close", "far"])
def test_rows_of_every_shape(V, kind):
    rng = np.random.default_rng(V + len(kind))
    z, u = shapes_of(rng, len(SETTINGS), V, kind), rng.random(len(SETTINGS))
    u[3], u[7] = 0.0, 1 - 2.0 ** -53
    check_sample(z, SETTINGS, u, run_sample(z, SETTINGS, u))


@pytest.mark.parametrize("V", [3001, 20011, 151936])
def test_as_many_as_are_listed(V):
    """Runs of large values that the row's sample sees whole, and a top-k of
    just as many: the list ends where the filter does."""
    rng = np.random.default_rng(V)
    z = np.zeros((6, V), np.float32)
    for i, n in enumerate((1, 1, 2, 3, 40, 64)):
        z[i, :n] = 30 + rng.permutation(n)
    s = [(1.0, 1, 1.0, 0.0), (1.0, 1, 0.5, 0.0), (1.0, 2, 1.0, 1e-30), (1.0, 3, 0.99, 0.0), (9.0, 40, 1.0, 0.0), (9.0, 64, 1.0, 0.01)]
    u = rng.random(6)
    got = run_sample(z, s, u)
    check_sample(z, s, u, got)
    assert (got["kept"] != -np.inf).sum(1)[[0, 2, 4]].tolist() == [1, 2, 40]


def test_more_rows_than_are_under_way_at_once():
    """Flat rows, failing ones and others in every part of the call."""
    rng = np.random.default_rng(1)
    rows, V = 700, 5003
    z = logits_of(rng, rows, V, "peaked")
    z[::3] = logits_of(rng, len(z[::3]), V, "flat")
    z[5::97, 11] = np.nan
    s, u = draw_settings(rng, rows, V), rng.random(rows)
    got = run_sample(z, s, u)
    check_sample(z, s, u, got)
    for i in (0, 255, 256, 511, 699):
        one = run_sample(z[i:i + 1], s[i:i + 1], u[i:i + 1])
        for n in one:
            assert one[n][0].tobytes() == got[n][i].tobytes()


def test_offsets_past_32_bits():
    """Logits whose rows lie 2^30 values apart, and outputs of more than 2^31."""
    t = torch()
    V, ld = 40001, 1 << 30
    far = t.empty(2 * ld + V, device="cuda")
    z = far.as_strided((3, V), (ld, 1))
    rng = np.random.default_rng(3)
    rows = logits_of(rng, 3, V, "peaked")
    z.copy_(dev(rows))
    u = rng.random(3)
    out = dict(tokens=t.zeros(3, dtype=t.int32, device="cuda"), probs=t.zeros((3, V), device="cuda"))
    sv.sample(z, sv.sampling_params(0.9, 50, 0.9), dev(u), out["tokens"], sv.sample_workspace(3, V), probs=out["probs"])
    want = run_sample(rows, [(0.9, 50, 0.9, 0.0)], u)
    assert np.array_equal(host(out["tokens"]), want["tokens"]) and np.array_equal(host(out["probs"]), want["probs"])
    del far, z
    V, n = 1 << 24, 130
    z, probs = t.zeros((n, V), device="cuda"), t.full((n, V), 7.0, device="cuda")
    for i, row in ((0, 5), (127, 9), (128, 77), (129, V - 1)):
        z[i, row] = 30.0
    tok, u = t.zeros(n, dtype=t.int32, device="cuda"), t.full((n,), 0.5, dtype=t.float64, device="cuda")
    sv.sample(z, sv.sampling_params(1.0, 1), u, tok, sv.sample_workspace(n, V), probs=probs)
    tok = host(tok)
    for i, row in ((0, 5), (127, 9), (128, 77), (129, V - 1), (64, 0)):
        assert tok[i] == row and probs[i, row].item() == 1.0 and probs[i].count_nonzero().item() == 1


def test_samples_side_by_side():
    """Calls on two streams and in two graphs, with a workspace each."""
    t = torch()
    rng = np.random.default_rng(4)
    V = 50021
    z = [logits_of(rng, 9, V, k) for k in ("peaked", "flat")]
    s = [draw_settings(rng, 9, V) for _ in z]
    u = [rng.random(9) for _ in z]
    want = [run_sample(*a) for a in zip(z, s, u)]
    dz, du = [dev(a) for a in z], [dev(a) for a in u]
    p = [sv.sampling_params(*(np.asarray(a)[:, i].astype(np.int64 if i == 1 else float) for i in range(4))) for a in s]
    tok = [t.zeros(9, dtype=t.int32, device="cuda") for _ in z]
    kept = [t.zeros((9, V), device="cuda") for _ in z]
    ws = [sv.sample_workspace(9, V) for _ in z]
    streams = [t.cuda.Stream() for _ in z]
    graphs = [t.cuda.CUDAGraph() for _ in z]
    t.cuda.synchronize()

    def check():
        t.cuda.synchronize()
        for i in range(2):
            assert np.array_equal(host(tok[i]), want[i]["tokens"])
            assert host(kept[i]).tobytes() == want[i]["kept"].tobytes()
            tok[i].zero_()
            kept[i].zero_()
        t.cuda.synchronize()

    for _ in range(10):
        for i, stream in enumerate(streams):
            sv.sample(dz[i], p[i], du[i], tok[i], ws[i], kept=kept[i], stream=stream)
    check()
    for i, g in enumerate(graphs):
        with t.cuda.graph(g):
            sv.sample(dz[i], p[i], du[i], tok[i], ws[i], kept=kept[i])
    for _ in range(5):
        for g, stream in zip(graphs, streams):
            with t.cuda.stream(stream):
                g.replay()
        check()


def test_norm_past_32_bits():
    """More than 2^31 elements, in place; the rows at the ends and about the
    2^31st element equal the same rows alone."""
    t = torch()
    rows, K = 65600, 32768
    x = t.full((rows, K), 0.5, device="cuda")
    at = [0, 1, 65535, 65536, 65599]
    some = t.randn((len(at), K), device="cuda")
    q = t.zeros((rows, K), dtype=t.int8, device="cuda")
    d, ss = t.zeros((rows, K // 32), device="cuda"), t.zeros((rows, K // 32), device="cuda")
    s16 = t.zeros((rows, K // 16), dtype=t.int32, device="cuda")
    gamma = t.randn(K, device="cuda")
    for fold in (False, True):
        want = norm_buffers(len(at), K)
        want["y"] = None
        for i, r in enumerate(at):
            x[r] = some[i]
        sv.add_norm_q8(some, some, gamma=gamma, fold=fold, **want)
        sv.add_norm_q8(x, x, gamma=gamma, fold=fold, sum=x, q=q, d=d, s16=s16, sumsq=ss)
        for got, name in ((x, "sum"), (q, "q"), (d, "d"), (s16, "s16"), (ss, "sumsq")):
            assert t.equal(got[at], want[name]), name
        assert (x[2:65535:257] == (2.0 if fold else 1.0)).all()


def test_norms_side_by_side():
    """On two streams, and captured and replayed with eager work between."""
    t = torch()
    x, dl = t.randn((40, 2560), device="cuda"), t.randn((40, 2560), device="cuda")
    a, b, g = norm_buffers(40, 2560), norm_buffers(40, 2560), t.cuda.CUDAGraph()
    want = norm_buffers(40, 2560)
    streams = [t.cuda.Stream(), t.cuda.Stream()]
    t.cuda.synchronize()
    for _ in range(10):
        for stream, out in zip(streams, (a, b)):
            sv.add_norm_q8(x, dl, stream=stream, **out)
    t.cuda.synchronize()
    sv.add_norm_q8(x, dl, **want)
    for n in want:
        assert t.equal(a[n], want[n]) and t.equal(b[n], want[n])
    with t.cuda.graph(g):
        sv.add_norm_q8(x, dl, **a)
    for _ in range(4):
        x.normal_()
        sv.add_norm_q8(x, dl, **want)
        g.replay()
        t.cuda.synchronize()
        for n in want:
            assert t.equal(a[n], want[n])


@pytest.mark.parametrize("K", [2560, 12320])
def test_rows_that_are_not_finite(K):
    """An infinity or a NaN stays in its row; the largest finite values, whose
    squares are not finite, too."""
    t = torch()
    rng = np.random.default_rng(K)
    x = rng.standard_normal((6, K)).astype(np.float32)
    x[1, 40], x[3, K - 1], x[4, 7] = np.nan, np.inf, 3e38
    bad, out, want = dev(x), norm_buffers(6, K), norm_buffers(6, K)
    sv.add_norm_q8(bad, **out)
    x[[1, 3, 4]] = 1
    sv.add_norm_q8(dev(x), **want)
    for n in want:
        assert t.equal(out[n][[0, 2, 5]], want[n][[0, 2, 5]]), n
    assert np.array_equal(host(out["sum"])[3, :-1], host(bad)[3, :-1])


@pytest.mark.parametrize("kind", ["f16", "bf16", "i8"])
def test_a_sequence_twice_and_two_plans_at_once(kind):
    t = torch()
    f = Forks(dict(f16=km.F16, bf16=km.BF16, i8=km.I8)[kind], 2, 5, 128, 64, 900, [70, 5, 33, 12], 3, mode=2, rot=64)
    same = f.seq[[0, 1, 1, 3]].contiguous()
    want = [f.run(f.plan(0, 256)), f.run(f.plan(0, 256), seq=same)]
    plans = [f.plan(f.shared, 256), f.plan(f.shared, 256)]
    seqs = [f.seq, same]
    for _ in range(2):
        for i in range(2):
            assert np.array_equal(f.run(plans[i], seq=seqs[i]), want[i])
    outs = [t.zeros((f.B, f.M, 10, 128), device="cuda") for _ in plans]
    streams = [t.cuda.Stream() for _ in plans]
    t.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            plans[i].run(0, f.q, outs[i], seq=seqs[i], n_new=f.n_arg, tree=f.tree, rope=f.rope, stream=streams[i])
    t.cuda.synchronize()
    for i in range(2):
        assert np.array_equal(host(outs[i]), want[i])
    assert f.kv.status() == 0


def test_shared_slots_past_the_sequences_and_one_sequence():
    """All that a sequence holds is shared; a batch of one; one slot alone."""
    for own, prompt in (([0, 0, 0], 512), ([4], 640), ([0, 1], 64)):
        f = Forks(km.F16, 2, 3, 64, 64, prompt, own, 2)
        for shared in (0, 1, f.shared // 2, f.shared):
            assert np.array_equal(f.run(f.plan(shared, 128)), f.run(f.plan(0, 128))), (own, shared)


@pytest.mark.parametrize("rows,V", [(1, 2561), (5, 50021), (13, 151936), (14, 151936), (64, 30000), (65, 30000)])
def test_flat_rows_in_one_launch_and_in_two(rows, V):
    """About the number of chunks up to which both passes over flat rows are
    one launch; a row's bits are the same either way."""
    rng = np.random.default_rng(rows)
    z, u = logits_of(rng, rows, V, "flat"), rng.random(rows)
    s = [SETTINGS[i % 10] for i in range(rows)]
    got = run_sample(z, s, u)
    check_sample(z, s, u, got)
    many = run_sample(np.concatenate([z] * 20), s * 20, np.concatenate([u] * 20))
    for n in got:
        assert got[n].tobytes() * 20 == many[n].tobytes(), n
