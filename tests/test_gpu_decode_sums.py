"""Sampling where a row's sum of weights is hard to form: logits that are
large against the temperature, with the row's largest value among the first
ones (which every sample of a row holds) or everywhere."""

import numpy as np
import pytest

import decode_model as dm
import speculative_decoding_verification_amd as sv
from gpu_util import dev, host, torch
from test_gpu_decode import check_sample, run_sample

pytestmark = pytest.mark.gpu

LOWEST = float(np.finfo(np.float32).min)


def rows_below(rng, tops, V, how):
    """Rows whose largest values are `tops`: `alone` the fifth element, far
    above the others; `twice` that and the last one; `close` all within twenty
    roundings of it; `all` nothing else."""
    z = np.empty((len(tops), V), np.float32)
    for i, top in enumerate(tops):
        top = np.float32(top)
        if how in ("alone", "twice"):
            with np.errstate(over="ignore"):
                z[i] = np.maximum(top - (np.abs(top) + 1) * rng.uniform(0.2, 0.9, V), LOWEST)
        elif how == "close":
            step = np.nextafter(np.abs(top), np.float32(0))
            z[i] = np.maximum(np.float64(top) - (np.float64(np.abs(top)) - step) * rng.integers(1, 20, V), LOWEST)
        else:
            z[i] = top
        z[i, 5] = top
        if how == "twice":
            z[i, V - 1] = top
    return z


def check_rows(rng, tops, V, how, temperatures):
    z = np.repeat(rows_below(rng, tops, V, how), 2 * len(temperatures), 0)
    s = [(t, 0, p, 0.0) for t in temperatures for p in (1.0, 0.9)] * len(tops)
    u = rng.random(len(s))
    check_sample(z, s, u, run_sample(z, s, u))


@pytest.mark.parametrize("V", [3001, 20011, 151936])
@pytest.mark.parametrize("how", ["alone", "twice", "close", "all"])
def test_temperatures_next_to_zero(V, how):
    tops = [21.0, 13.0, 20.1] if V > 100000 else [21.0, 13.0, 11.0, 19.0, 20.1, 7.25, 12.7, 15.3, -3.25, -20.1, 0.0]
    ts = [1e-6, 1e-8, 1e-10, 1e-12, 1e-14, 1e-15, 1e-16, 1e-17, 1e-20, 1e-30, 1e-38]
    check_rows(np.random.default_rng(V), tops, V, how, ts[::2] if V > 100000 else ts)


@pytest.mark.parametrize("V", [3001, 20011, 151936])
@pytest.mark.parametrize("how", ["alone", "twice", "close", "all"])
def test_logits_of_any_magnitude(V, how):
    tops = [1e10, -1e9, LOWEST] if V > 100000 else [1e6, -1e6, 1e9, -1e9, 1e10, 1e13, -1e15, 1e16, -1e17, 1e30, 3e38, -3e38, LOWEST]
    check_rows(np.random.default_rng(V + 1), tops, V, how, [0.7, 1.0, 300.0])


@pytest.mark.parametrize("V", [3001, 151936])
def test_rows_of_one_value_are_uniform(V):
    """Every token is as likely as any other, whatever the value: kept whole
    without a filter, the first ones up to top-p of them, and the token u
    says."""
    tops, u = [LOWEST, -1e10, 1e10, 20.1], [0.0, 0.37, 0.5, 0.999]
    z = np.repeat(np.float32(tops)[:, None], V, 1)
    for t in (0.7, 1e-12, 1e-17):
        got = run_sample(z, [(t, 0, 1.0, 0.0)], u)
        assert (got["kept"] == z).all() and (np.abs(got["probs"] * np.float64(V) - 1) <= 2.0 ** -23).all()
        assert (np.abs(got["tokens"] - np.floor(np.multiply(u, V))) <= 1).all()
        got = run_sample(z, [(t, 0, 0.25, 0.0)], u)
        n = -(-V // 4)
        assert ((got["kept"] != -np.inf).sum(1) == n).all() and (got["kept"][:, :n] == z[:, :n]).all()


@pytest.mark.parametrize("V,at", [(67 * 8192, (64, 65)), (1 << 24, (256, 260)), (1 << 24, (2040, 2044)), (1 << 24, (2044, 2045))])
def test_the_last_tokens_of_a_masked_row(V, at):
    """A certain token and, in two later pieces of 8192, one each of weight
    0.4 * 2^-52, which sums lose or not by their order; all behind is masked.
    u next to 1 gives one of the three, never a masked token."""
    t = torch()
    z = t.full((1, V), -np.inf, device="cuda")
    z[0, :8192] = -5000.0                       # finite, and of no weight
    able = [5] + [8192 * c + 100 for c in at]
    z[0, able[0]] = 0.0
    z[0, able[1:]] = -36.96
    tok = t.zeros(1, dtype=t.int32, device="cuda")
    u = t.full((1,), 1 - 2.0 ** -53, dtype=t.float64, device="cuda")
    sv.sample(z, sv.sampling_params(1.0), u, tok, sv.sample_workspace(1, V))
    assert tok.item() in able
    u.fill_(0.5)
    sv.sample(z, sv.sampling_params(1.0), u, tok, sv.sample_workspace(1, V))
    assert tok.item() == 5


def test_a_share_of_weights_below_half_a_step():
    """One token of weight 1 and 2^22 - 1 just below half a step, whose sum
    passes what top-p leaves: by the sum of the weights as they are nearly all
    are kept, and as the steps do not reach it, all."""
    V = 1 << 22
    z = np.full((1, V), -29.2, np.float32)
    assert np.exp(-29.2) < 2.0 ** -(dm.steps(V) + 1)
    z[0, 77] = 0.0
    s, u = [(1.0, 0, 1 - 2.0 ** -24, 0.0)], [0.9]
    got = run_sample(z, s, u)
    check_sample(z, s, u, got)
    assert got["tokens"].tolist() == [77] and (got["kept"] == z).all()
    s = [(1.0, 0, 0.999, 0.0)]
    got = run_sample(z, s, u)
    assert (got["kept"] != -np.inf).sum() == 1 and got["kept"][0, 77] == 0.0
