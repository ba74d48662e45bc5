"""The cache's wrapper without a GPU: what it refuses before any tensor is
looked at by a call."""

import pytest
import torch

import speculative_decoding_verification_amd as sv
from speculative_decoding_verification_amd.kv import KvCache


class Recorded(KvCache):
    """A wrapper without buffers, that records the calls it would make."""

    def __init__(self, seqs):
        self.seqs, self._torch, self._struct, self.calls = seqs, torch, sv.KvBatch, []
        self._lib = type("Lib", (), {"sv_kv_commit": None})

    def _tensor(self, t, name, dtype, shape=None):
        return None if t is None else 256

    def _call(self, fn, *args, stream=None):
        self.calls.append(args)


@pytest.mark.parametrize("seqs,shape", [
    (2, ()), (3, (2,)), (3, (4,)), (2, (1, 5)), (2, (3, 5)), (2, (2, 0)), (2, (0,)), (2, (2, 1, 1)), (1, (0,)),
    (1, (1, 1, 1)), (1, (2, 5))])
def test_accepted_counts_of_other_shapes(seqs, shape):
    """A count for each sequence, or nothing is enqueued."""
    kv = Recorded(seqs)
    with pytest.raises(sv.SpecVerifyError):
        kv.commit(4, torch.zeros(shape, dtype=torch.int32))
    assert not kv.calls


@pytest.mark.parametrize("seqs,shape,stride", [
    (3, (3,), 1), (3, (3, 1), 1), (3, (3, 6), 6), (1, (6,), 1), (1, (1,), 1), (1, (1, 6), 6), (1, (), 1)])
def test_accepted_counts(seqs, shape, stride):
    kv = Recorded(seqs)
    kv.commit(4, torch.zeros(shape, dtype=torch.int32))
    assert len(kv.calls) == 1 and kv.calls[0][2] == stride
