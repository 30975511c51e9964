"""The weight and eviction calls refuse outputs that share memory with what
the same call still reads (on the host, before any launch; no GPU)."""
import ctypes
import itertools

import pytest
import torch

from sequence_sharded_decode_gb300 import dcp
from test_compress_abi import GOOD, _desc, lib  # noqa: F401  (fixture)

# the addresses are made up: a call that were let through must not find a GPU
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")

B, N, HKV, CAP = 3, 2, 2, 100
ROWS = B * HKV * CAP * 4
SIZES = dict(lens=4 * B, starts=4 * B * N, keep=4 * B * N, mi=ROWS, pi=ROWS, known=4 * B, total=4 * B,
             mo=ROWS, po=ROWS, ns=4 * B * N, nl=4 * B, ws=1 << 16)
INPUTS, OUTPUTS = ("lens", "starts", "keep", "mi", "pi", "known", "total"), ("mo", "po", "ns", "nl", "ws")


def _evict(lib, **at):
    """Every array at an address of its own, far from the others, unless given."""
    a = {k: 1 << 20 | i << 16 for i, k in enumerate(SIZES)}
    a.update(at)
    shards = (dcp._Shard * 2)(GOOD, GOOD)
    return lib.dcp_kv_evict(ctypes.byref(_desc().c()), shards, N, a["lens"], a["starts"], B, a["keep"], 1, 1, a["mi"],
                            a["pi"], a["known"], a["total"], CAP, a["mo"], a["po"], a["ns"], a["nl"], a["ws"],
                            SIZES["ws"], None, None)


def _place(k):
    return 1 << 20 | list(SIZES).index(k) << 16


@pytest.mark.parametrize("out,other", [(o, x) for o in OUTPUTS for x in INPUTS]
                         + list(itertools.combinations(OUTPUTS, 2)))
def test_eviction_refuses_shared_memory(lib, out, other):  # noqa: F811
    if out == "ws" or other == "ws":     # the workspace has to stay aligned: the other one moves into it
        out, other = ("ws", out) if other == "ws" else (out, other)
        moved, base = other, _place("ws")
        assert _evict(lib, **{moved: base}) == dcp.DCP_ERR_INVALID_ARG
        assert _evict(lib, **{moved: base + SIZES["ws"] - 4}) == dcp.DCP_ERR_INVALID_ARG
        return
    assert _evict(lib, **{out: _place(other)}) == dcp.DCP_ERR_INVALID_ARG
    # the last word of the other array, and the last word of this one
    assert _evict(lib, **{out: _place(other) + SIZES[other] - 4}) == dcp.DCP_ERR_INVALID_ARG
    assert _evict(lib, **{out: _place(other) - SIZES[out] + 4}) == dcp.DCP_ERR_INVALID_ARG


def _mass(lib, q=1 << 20, lens=2 << 20, starts=3 << 20, lse=4 << 20, mi=None, mo=5 << 20, cap=CAP):
    shards = (dcp._Shard * 2)(GOOD, GOOD)
    return lib.dcp_attention_mass(ctypes.byref(_desc().c()), q, shards, N, lens, starts, B, 1, lse, mi, mo, cap, None, None)


@pytest.mark.parametrize("kw", [dict(mi=(5 << 20) + 4), dict(mi=(5 << 20) - 4), dict(mi=(5 << 20) + ROWS - 4),
                                dict(q=5 << 20), dict(lse=(5 << 20) + ROWS - 4), dict(lens=(5 << 20) + 8),
                                dict(starts=(5 << 20) + 8), dict(lse=(5 << 20) + (1 << 40), cap=1 << 62)])
def test_weights_refuse_shared_memory(lib, kw):  # noqa: F811
    """Masses may be added to in place, at the same address; anything else that overlaps them is read while it is written."""
    assert _mass(lib, **kw) == dcp.DCP_ERR_INVALID_ARG
