"""Whether the rule shares: a sequence that does not hold a shared page is
told by the attention that reads shared slots once, and by no other."""

import numpy as np
import pytest

import speculative_decoding_verification_amd as sv
from gpu_util import host
from test_gpu_shared import KINDS, Forks

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,heads,group,dim,page,prompt,own,M,shares", [
    ("bf16", 8, 5, 128, 64, 4096, [1] * 32, 1, True), ("f16", 8, 5, 128, 64, 4096, [1] * 16, 5, True),
    ("i8", 4, 4, 64, 64, 8192, [1] * 32, 1, True), ("f16", 4, 5, 128, 64, 960, [60, 20, 40, 1], 1, False),
    ("bf16", 4, 5, 128, 64, 960, [60, 20, 40, 1], 1, False)])
def test_the_rule_shares_where_it_pays(kind, heads, group, dim, page, prompt, own, M, shares):
    f = Forks(KINDS[kind], heads, group, dim, page, prompt, own, M, mode=2, rot=dim)
    assert f.shared == prompt
    plan = f.plan(f.shared)
    want = f.run(plan)
    f.check(want, 1 << 14)
    assert f.kv.status() == 0
    # the first two pages of the last sequence change places
    row = int(host(f.seq)[-1])
    f.kv.table[row, :2] = f.kv.table[row, :2].flip(0).clone()
    got = f.run(plan)
    assert np.array_equal(got[:-1], want[:-1])
    if shares:
        assert np.isnan(got[-1]).all() and f.kv.status() == sv.SV_KV_NOT_SHARED
    else:
        assert np.isfinite(got[-1]).all() and f.kv.status() == 0
