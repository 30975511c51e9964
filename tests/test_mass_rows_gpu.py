"""Query rows that are to add nothing to the attention weight (lse -inf), whatever they hold."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from compress_helpers import Cache, as_cached, check_mass, normal_rows, queries
from helpers import f64
from sequence_sharded_decode_gb300 import dcp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [math.nan, math.inf, 3e38])
@pytest.mark.parametrize("kv,hq,hkv,d,bs,J", [
    ("bf16", 8, 2, 64, 16, 1), ("fp8", 8, 2, 64, 16, 1), ("mxfp4", 4, 1, 128, 16, 2),     # up to 16 rows
    ("bf16", 32, 1, 64, 16, 1), ("bf16", 24, 1, 128, 16, 1), ("bf16", 8, 2, 128, 16, 40),  # more
    ("fp8", 32, 1, 128, 16, 2), ("mxfp4", 40, 2, 64, 16, 3),
    ("bf16", 128, 1, 576, 64, 1), ("fp8", 128, 1, 576, 64, 2)])
def test_excluded_rows_may_hold_anything(kv, hq, hkv, d, bs, J, bad):
    lens = [300, 70]
    rows = normal_rows(lens, hkv, d, 61)
    c = Cache(kv, lens, hq, hkv, d, bs, 2, rows)
    q = queries(2, J, hq, d, 13)
    keys = [as_cached(kv, r[0]) for r in rows]
    lse = torch.stack([torch.tensor(np.maximum(O.mtp_attention(f64(q[b]), keys[b], keys[b], c.desc.scale, n)[1], -1e3),
                                    dtype=torch.float32) for b, n in enumerate(lens)])
    out_rows = torch.zeros(2, J, hq, dtype=torch.bool)
    out_rows[:, J // 2, ::3] = True
    out_rows[1, :, -1] = True
    lse[out_rows] = -math.inf
    clean = q.clone()
    q[out_rows] = bad
    q[0, J // 2, 0, 1::2] *= -1
    mass = torch.full((2, hkv, 300), 7.0, device="cuda")
    dcp.dcp_attention_mass(c.desc, q.cuda(), c.shards, c.seq_lens, c.starts, lse.cuda(), mass, err=c.err)
    assert c.flag() == 0
    for b, n in enumerate(lens):
        w = O.attention_mass(f64(clean[b]), keys[b], c.desc.scale, n, lse[b].numpy().astype(np.float64))
        check_mass(mass[b, :, :n].cpu().numpy(), w, f64(clean[b]), keys[b], c.desc.scale, None, (b, bad))
        assert (mass[b, :, n:] == 7).all()
