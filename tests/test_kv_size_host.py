"""Sizes and numbers past what the arithmetic holds are refused, not wrapped."""

import ctypes
import os

import pytest

import speculative_decoding_verification_amd as sv
from test_kv_host import F, batch, cache, refused

pytestmark = pytest.mark.skipif(not os.path.exists(sv.LIB_PATH), reason="libspecverify.so not built")


@pytest.mark.parametrize("layers,heads,n_pages", [
    (1638, 3001, 14315282),   # 2^64 bytes and 590348288
    (1024, 4096, 1 << 24),    # 2^64
    (2047, 4096, 1 << 24), (64, 512, 1 << 15)])
def test_pools_past_all_memory(layers, heads, n_pages):
    L, r = sv.lib(), ctypes.byref
    kv = cache(layers=layers, heads=heads, n_pages=n_pages, dim=256, page=256)
    assert layers * heads * n_pages * 8 * 128 * 256 >= 1 << 48
    assert L.sv_kv_data_bytes(r(kv)) == 0
    refused(L.sv_kv_init(r(kv), None), sv.SV_ERR_SHAPE)
    refused(L.sv_kv_append(r(kv), 0, r(batch()), F, F, None, None), sv.SV_ERR_SHAPE)
    refused(L.sv_kv_compact(r(kv), F, 1 << 40, None), sv.SV_ERR_SHAPE)


def test_the_largest_pool():
    L, r = sv.lib(), ctypes.byref
    kv = cache(layers=64, heads=512, n_pages=(1 << 15) - 1, dim=256, page=256)
    assert L.sv_kv_data_bytes(r(kv)) == (1 << 48) - (1 << 33)
    assert L.sv_kv_data_bytes(r(cache(layers=4096, heads=4096))) == 0   # no call takes it


@pytest.mark.parametrize("scale", [2.35e38, 2.4e38, 3e38, 3.4e38])
def test_scales_that_base_two_makes_infinite(scale):
    L, kv, b, r = sv.lib(), cache(), batch(), ctypes.byref
    a = sv.KvAttn(40, scale, 0, 0, 0, 0, None)
    refused(L.sv_kv_attention(r(kv), 0, r(b), r(a), F, F, None, F, 1 << 40, None), sv.SV_ERR_ARG)
    assert L.sv_kv_attention_workspace_bytes(r(kv), r(b), r(a)) == 0
    a = sv.KvAttn(40, 2.3e38, 0, 0, 0, 0, None)
    assert L.sv_kv_attention_workspace_bytes(r(kv), r(b), r(a)) > 0
