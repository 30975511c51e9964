"""The eviction binding refuses what the library could not see: a workspace on
another device, counts that do not fit its integers (no GPU)."""
import types

import pytest
import torch

from sequence_sharded_decode_gb300 import dcp


@pytest.fixture
def evict(monkeypatch):
    """dcp_kv_evict with every other check satisfied; the library call is recorded, not made."""
    calls = []
    monkeypatch.setattr(dcp, "_check", lambda *a, **k: None)
    monkeypatch.setattr(dcp, "_check_shape", lambda *a, **k: None)
    monkeypatch.setattr(dcp, "_cache", lambda *a, **k: None)
    monkeypatch.setattr(dcp, "_stream", lambda s: 0)
    monkeypatch.setattr(dcp, "load", lambda: types.SimpleNamespace(dcp_kv_evict=lambda *a: calls.append(a) or 0))
    desc = dcp.AttnDesc(dcp.DCP_KIND_GQA, 8, 2, 64, 64, 16, 0.125)

    def tensor(*shape):
        return types.SimpleNamespace(shape=shape, dim=lambda: len(shape), data_ptr=lambda: 16, numel=lambda: 1 << 20,
                                     device=torch.device("cuda", 0))

    def call(n_sink=1, n_recent=1, device=0):
        ws = tensor(1 << 20)
        ws.device = torch.device("cuda", device)
        rows = tensor(1, 2, 10)
        dcp.dcp_kv_evict(desc, [None], tensor(1), tensor(1, 1), tensor(1, 1), n_sink, n_recent, rows, rows, rows,
                         tensor(1, 1), tensor(1), ws)
        return calls
    return call


def test_a_good_call_reaches_the_library(evict):
    assert len(evict()) == 1 and len(evict(n_sink=2 ** 31 - 1, n_recent=0)) == 2


def test_a_workspace_on_another_device_is_refused(evict):
    with pytest.raises(ValueError, match="workspace"):
        evict(device=1)


@pytest.mark.parametrize("kw", [dict(n_sink=2 ** 31), dict(n_recent=2 ** 32 + 3), dict(n_sink=-2 ** 32)])
def test_counts_beyond_int32_are_refused(evict, kw):
    with pytest.raises(ValueError, match="n_sink|n_recent"):
        evict(**kw)
