"""Attention through block tables with missing entries, over every cache type:
the tokens of a missing block count as not there, wherever in the sequence it
lies, and the flag is raised."""
import numpy as np
import pytest
import torch

import oracle as O
from compress_helpers import Cache, as_cached, normal_rows, queries, score_error
from helpers import f64
from sequence_sharded_decode_gb300 import dcp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [0.01, 1.0, 30.0])
@pytest.mark.parametrize("gone", ["first", "many", "last", "all", "scattered"])
@pytest.mark.parametrize("kv,hq,hkv,d,bs,J", [("mxfp4", 8, 2, 64, 16, 1), ("mxfp4", 16, 1, 128, 16, 1), ("mxfp4", 8, 1, 128, 32, 4),
                                              ("fp8", 8, 2, 64, 16, 1), ("fp8", 16, 1, 128, 16, 2), ("fp8", 128, 1, 576, 64, 1),
                                              ("bf16", 8, 2, 64, 16, 1), ("bf16", 16, 1, 128, 16, 2), ("bf16", 128, 1, 576, 64, 2)])
def test_attention_without_some_blocks(kv, hq, hkv, d, bs, J, gone, size):
    n, shards = 700, 2
    rows = normal_rows([n], hkv, d, 91)
    c = Cache(kv, [n], hq, hkv, d, bs, shards, rows)
    blocks = -(-350 // bs)
    which = {"first": [0], "many": list(range(min(blocks - 1, 160 // bs + 1))), "last": [blocks - 1],
             "all": list(range(blocks)), "scattered": list(range(1, blocks, 3))}[gone]
    there = np.ones(n, dtype=bool)
    for i, shard in enumerate(c.shards):
        for k, b in enumerate(which):
            shard.block_table[0, b] = -1 if k % 2 else 1 << 20
            there[350 * i + b * bs:min(350 * i + (b + 1) * bs, 350 * (i + 1))] = False
    q = queries(1, J, hq, d, 17, size=size)
    o, lse = c.attend(q.cuda())
    assert c.flag() == dcp.DCP_DEVERR_BLOCK_RANGE
    K = as_cached(kv, rows[0][0])
    V = K[..., :512] if d == 576 else as_cached(kv, rows[0][1])
    for j, lim in enumerate(O.mtp_limits(n, J)):
        seen = np.nonzero(there[:lim])[0]
        got, l = o[0, j].cpu().numpy(), lse[0, j].cpu().numpy()
        if not len(seen):
            assert (got == 0).all() and np.isneginf(l).all()
            continue
        ro, rl = O.attention(f64(q[0, j]), K[seen], V[seen], c.desc.scale, 0, len(seen))
        ds = score_error(f64(q[:1, j]), K[seen], c.desc.scale)
        rel = 2 * np.expm1(ds) + (2.0 ** -10 if kv == "fp8" else 2.0 ** -15) + 2.0 ** -19 + (n + 8) * 2.0 ** -23
        assert (np.abs(got - ro) <= rel * np.abs(V).max()).all(), (gone, np.abs(got - ro).max(), rel)
        assert np.abs(l - rl).max() <= ds + (n + 8) * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -22 * np.abs(rl).max()
