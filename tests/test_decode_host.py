"""What sampling, the residual's norm and attention over shared slots refuse,
without a GPU; and the models of their tests on values worked out by hand."""

import ctypes
import os

import numpy as np
import pytest

import decode_model as dm
import speculative_decoding_verification_amd as sv

needs_library = pytest.mark.skipif(not os.path.exists(sv.LIB_PATH), reason="libspecverify.so not built")
FAKE = 1 << 44


def at(i, off=0):
    """Addresses far apart: buffers that do not overlap."""
    return ctypes.c_void_p(FAKE + (i << 38) + off)


def refused(rc, code):
    assert rc == code, (rc, sv.lib().sv_last_error())
    assert sv.lib().sv_last_error()


def norm(x=at(0), delta=at(1), rows=5, K=64, gamma=at(2), eps=1e-6, fold=0, sum=at(3), y=at(4), q=at(5), d=at(6),
         s16=at(7), sumsq=at(8)):
    return sv.lib().sv_add_norm_q8(x, delta, rows, K, gamma, eps, fold, sum, y, q, d, s16, sumsq, None)


@needs_library
@pytest.mark.parametrize("change,code", [
    (dict(x=None), sv.SV_ERR_ARG), (dict(y=None, q=None, d=None, s16=None, sumsq=None), sv.SV_ERR_ARG),
    (dict(q=None), sv.SV_ERR_ARG), (dict(d=None), sv.SV_ERR_ARG), (dict(s16=None), sv.SV_ERR_ARG),
    (dict(sumsq=None), sv.SV_ERR_ARG), (dict(fold=2), sv.SV_ERR_ARG), (dict(fold=-1), sv.SV_ERR_ARG),
    (dict(fold=1), sv.SV_ERR_ARG), (dict(fold=1, q=None, d=None, s16=None, sumsq=None), sv.SV_ERR_ARG),
    (dict(eps=-1e-6), sv.SV_ERR_ARG), (dict(eps=float("nan")), sv.SV_ERR_ARG), (dict(eps=float("inf")), sv.SV_ERR_ARG),
    (dict(K=0), sv.SV_ERR_SHAPE), (dict(K=48), sv.SV_ERR_SHAPE), (dict(K=-32), sv.SV_ERR_SHAPE),
    (dict(K=32768 + 32), sv.SV_ERR_SHAPE), (dict(rows=0), sv.SV_ERR_SHAPE), (dict(rows=-1), sv.SV_ERR_SHAPE),
    (dict(rows=1 << 27), sv.SV_ERR_SHAPE), (dict(rows=1 << 62), sv.SV_ERR_SHAPE), (dict(x=at(0, 4)), sv.SV_ERR_ALIGN),
    (dict(delta=at(1, 8)), sv.SV_ERR_ALIGN), (dict(gamma=at(2, 4)), sv.SV_ERR_ALIGN), (dict(sum=at(3, 4)), sv.SV_ERR_ALIGN),
    (dict(y=at(4, 8)), sv.SV_ERR_ALIGN), (dict(q=at(5, 1)), sv.SV_ERR_ALIGN), (dict(d=at(6, 2)), sv.SV_ERR_ALIGN),
    (dict(s16=at(7, 1)), sv.SV_ERR_ALIGN), (dict(sumsq=at(8, 2)), sv.SV_ERR_ALIGN),
    (dict(y=at(0)), sv.SV_ERR_ARG), (dict(y=at(1)), sv.SV_ERR_ARG), (dict(sum=at(0, 16)), sv.SV_ERR_ARG),
    (dict(sum=at(1, 5 * 64 * 4 - 16)), sv.SV_ERR_ARG), (dict(sum=at(2)), sv.SV_ERR_ARG), (dict(q=at(0, 64)), sv.SV_ERR_ARG),
    (dict(y=at(3)), sv.SV_ERR_ARG), (dict(d=at(5, 4)), sv.SV_ERR_ARG), (dict(s16=at(6)), sv.SV_ERR_ARG),
    (dict(sumsq=at(7)), sv.SV_ERR_ARG)])
def test_norm_arguments(change, code):
    refused(norm(**change), code)


def take(logits=at(0), rows=4, V=1000, ld=1000, params=at(1), n_params=1, u=at(2), tokens=at(3), probs=at(4), kept=at(5),
         ws=at(6), n=None):
    n = sv.lib().sv_sample_workspace_bytes(4, 1000) if n is None else n
    return sv.lib().sv_sample(logits, rows, V, ld, params, n_params, u, tokens, probs, kept, ws, n, None)


@needs_library
@pytest.mark.parametrize("change,code", [
    (dict(logits=None), sv.SV_ERR_ARG), (dict(params=None), sv.SV_ERR_ARG), (dict(u=None), sv.SV_ERR_ARG),
    (dict(tokens=None, probs=None, kept=None), sv.SV_ERR_ARG), (dict(ws=None), sv.SV_ERR_ARG),
    (dict(n=0), sv.SV_ERR_WORKSPACE), (dict(rows=0), sv.SV_ERR_SHAPE), (dict(rows=65536), sv.SV_ERR_SHAPE),
    (dict(V=0), sv.SV_ERR_SHAPE), (dict(V=(1 << 24) + 1, ld=1 << 25), sv.SV_ERR_SHAPE), (dict(ld=999), sv.SV_ERR_SHAPE),
    (dict(ld=1 << 31), sv.SV_ERR_SHAPE), (dict(n_params=0), sv.SV_ERR_ARG), (dict(n_params=3), sv.SV_ERR_ARG),
    (dict(n_params=5), sv.SV_ERR_ARG), (dict(logits=at(0, 2)), sv.SV_ERR_ALIGN), (dict(params=at(1, 2)), sv.SV_ERR_ALIGN),
    (dict(u=at(2, 4)), sv.SV_ERR_ALIGN), (dict(tokens=at(3, 2)), sv.SV_ERR_ALIGN), (dict(probs=at(4, 1)), sv.SV_ERR_ALIGN),
    (dict(kept=at(5, 2)), sv.SV_ERR_ALIGN), (dict(ws=at(6, 128)), sv.SV_ERR_ALIGN), (dict(kept=at(0)), sv.SV_ERR_ARG),
    (dict(probs=at(0, 4 * 4 * 1000 - 4)), sv.SV_ERR_ARG), (dict(kept=at(4, 400)), sv.SV_ERR_ARG)])
def test_sample_arguments(change, code):
    refused(take(**change), code)


@needs_library
def test_sample_workspaces():
    L = sv.lib()
    for rows, V in ((0, 10), (65536, 10), (1, 0), (1, (1 << 24) + 1), (-1, 5)):
        assert L.sv_sample_workspace_bytes(rows, V) == 0
    for rows, V in ((1, 1), (65535, 1 << 24), (5, 151936)):
        assert L.sv_sample_workspace_bytes(rows, V) > 0
    # a workspace serves any smaller call
    for rows, V in ((256, 151936), (9, 40000), (1, 1 << 24)):
        most = L.sv_sample_workspace_bytes(rows, V)
        for r, v in ((1, V), (rows, 1), (rows // 2 + 1, V // 2 + 1), (1, 1), (rows, V - 1 or 1)):
            assert L.sv_sample_workspace_bytes(r, v) <= most
    with pytest.raises(sv.SpecVerifyError):
        sv.sample_workspace(0, 10, device="cpu")


def test_settings():
    p = sv.sampling_params(0.5, [0, 40, 7], 0.9, np.float32(0.25), device="cpu").numpy()
    assert p.shape == (3, 4) and p.dtype == np.int32
    assert p[:, 1].tolist() == [0, 40, 7]
    f = p.view(np.float32)
    assert (f[:, 0] == 0.5).all() and (f[:, 2] == np.float32(0.9)).all() and (f[:, 3] == 0.25).all()
    assert sv.sampling_params(device="cpu").numpy().view(np.float32)[0, [0, 2, 3]].tolist() == [1.0, 1.0, 0.0]
    for bad in (dict(temperature=[1.0, 2.0], top_k=[1, 2, 3]), dict(top_p=[[0.5]]), dict(top_p=[]), dict(top_k=40.5),
                dict(top_k=1 << 31), dict(top_k=[1, -(1 << 31) - 1])):
        with pytest.raises(sv.SpecVerifyError):
            sv.sampling_params(**bad, device="cpu")


def test_tensors_on_the_host_are_refused():
    import torch
    x = torch.zeros(2, 32)
    with pytest.raises(sv.SpecVerifyError):
        sv.add_norm_q8(x, y=torch.zeros(2, 32))
    with pytest.raises(sv.SpecVerifyError):
        sv.sample(x, sv.sampling_params(device="cpu"), torch.zeros(2, dtype=torch.float64),
                  torch.zeros(2, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8))


def cache(**change):
    d = dict(type=1, layers=1, heads=8, dim=128, page=64, n_pages=100, seqs=4, width=16)
    d.update(change)
    return sv.Kv(*d.values(), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE)


@needs_library
@pytest.mark.parametrize("shared,window,code", [(-1, 0, sv.SV_ERR_ARG), (16 * 64 + 1, 0, sv.SV_ERR_ARG), (64, 100, sv.SV_ERR_ARG),
                                                (1 << 30, 0, sv.SV_ERR_ARG)])
def test_shared_arguments(shared, window, code):
    F = ctypes.c_void_p(FAKE)
    kv, b, r = cache(), sv.KvBatch(4, 5, None, None, None), ctypes.byref
    a = sv.KvAttn(40, 0.1, window, 0, 0, 0, None)
    refused(sv.lib().sv_kv_attention_shared(r(kv), 0, r(b), r(a), shared, F, F, None, F, 1 << 40, None), code)
    assert sv.lib().sv_kv_attention_shared_workspace_bytes(r(kv), r(b), r(a), shared) == 0


@needs_library
def test_shared_sizes():
    """The workspace follows the chunk length alone; too many row groups of
    shared chunks are refused."""
    L, r = sv.lib(), ctypes.byref
    b = sv.KvBatch(4, 5, None, None, None)
    a = sv.KvAttn(40, 0.1, 0, 0, 0, 128, None)
    kv = cache()
    assert L.sv_kv_attention_shared_workspace_bytes(r(kv), r(b), r(a), 640) == L.sv_kv_attention_workspace_bytes(r(kv), r(b), r(a)) > 0
    kv = cache(width=1 << 12, seqs=4096)
    F, many = ctypes.c_void_p(FAKE), sv.KvBatch(4096, 16, None, None, None)
    a = sv.KvAttn(512, 0.1, 0, 0, 0, 128, None)
    refused(L.sv_kv_attention_shared(r(kv), 0, r(many), r(a), 1 << 17, F, F, None, F, 1 << 60, None), sv.SV_ERR_SHAPE)


def test_the_models():
    z = np.log(np.float32([4, 1, 2, 1])).astype(np.float32)
    keep = lambda *j: np.isin(np.arange(4), j)  # noqa: E731
    dm.check_kept(z, keep(0, 2, 1), (1.0, 3, 1.0, 0.0))     # equal ones: the lower index
    dm.check_kept(z, keep(0, 2), (1.0, 0, 0.7, 0.0))        # 4 + 2 of 8
    dm.check_kept(z, keep(0), (1.0, 2, 0.6, 0.0))           # 4 of 6
    dm.check_kept(z, keep(0, 2), (1.0, 0, 1.0, 0.3))
    dm.check_kept(z, keep(0), (0.0, 0, 1.0, 0.0))
    for wrong, params in ((keep(0, 2, 3), (1.0, 3, 1.0, 0.0)), (keep(0, 2, 1), (1.0, 0, 0.7, 0.0)),
                          (keep(0, 2), (1.0, 2, 0.6, 0.0)), (keep(0, 2, 1, 3), (1.0, 0, 1.0, 0.3))):
        with pytest.raises(AssertionError):
            dm.check_kept(z, wrong, params)
    dm.check_probs(z, keep(0, 2), np.float32([4 / 6, 0, 2 / 6, 0]), 1.0)
    dm.check_token(z, keep(0, 2), 0.5, 0, 1.0)
    dm.check_token(z, keep(0, 2), 0.7, 2, 1.0)
    for token, u in ((2, 0.5), (0, 0.7), (1, 0.7)):
        with pytest.raises(AssertionError):
            dm.check_token(z, keep(0, 2), u, token, 1.0)
    q, d, s = dm.codes(np.float32([[127.0, 2.5, -2.5, 0.4] + [0] * 28]), None)
    assert q[0, :4].tolist() == [127, 3, -3, 0] and d.tolist() == [[1.0]] and s.tolist() == [[127, 0]]
