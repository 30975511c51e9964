"""The decode loop with evictions, token by token: what every cached token has
been given by all the steps since it came, carried through the evictions in
64 bits; and one shard's range over the 4-bit cache."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from compress_helpers import Cache, as_cached, check_attention, check_mass, normal_rows, queries
from helpers import f64
from sequence_sharded_decode_gb300 import dcp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv,hq,hkv,d,bs,J", [("mxfp4", 8, 2, 64, 16, 1), ("mxfp4", 40, 2, 128, 16, 2),
                                              ("bf16", 32, 2, 128, 32, 1), ("bf16", 4, 2, 64, 16, 3),
                                              ("fp8", 8, 2, 64, 16, 1), ("fp8", 32, 1, 128, 16, 2),
                                              ("bf16", 128, 1, 576, 64, 1), ("fp8", 128, 1, 576, 64, 2)])
def test_every_tokens_mass_through_evictions(kv, hq, hkv, d, bs, J):
    lens, steps, shards, budget = [70, 45], 8, 2, 14
    rows = normal_rows([n + steps * J for n in lens], hkv, d, 81)
    c = Cache(kv, lens, hq, hkv, d, bs, shards, [(k[:n], None if v is None else v[:n]) for (k, v), n in zip(rows, lens)],
              spare=steps * J)
    cap = max(lens) + steps * J
    keys = [as_cached(kv, r[0]) for r in rows]
    held = [[list(range(n)) for _ in range(hkv)] for n in lens]      # text positions by cache index
    given = [np.zeros((hkv, n + steps * J)) for n in lens]           # by text position
    total, starts, seq_lens = list(lens), c.starts, c.seq_lens
    mass, pos, known = torch.full((2, hkv, cap), 7.0, device="cuda"), None, None
    for b, n in enumerate(lens):
        mass[b, :, :n] = 0
    every_q = []
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for step in range(steps):
        at = [len(held[b][0]) for b in range(2)]
        new = [range(total[b], total[b] + J) for b in range(2)]
        c.append([b for b in range(2) for _ in range(J)], [at[b] + j for b in range(2) for j in range(J)],
                 torch.cat([rows[b][0][list(new[b])] for b in range(2)]),
                 None if c.mla else torch.cat([rows[b][1][list(new[b])] for b in range(2)]), starts=starts)
        for b in range(2):
            for h in range(hkv):
                held[b][h] += list(new[b])
            total[b] += J
        seq_lens = seq_lens + J
        q = queries(2, J, hq, d, 90 + step, size=2.0)
        every_q.append(f64(q))
        _, lse = c.attend(q.cuda(), starts=starts, seq_lens=seq_lens)
        dcp.dcp_attention_mass(c.desc, q.cuda(), c.shards, seq_lens, starts, lse, mass, mass_in=mass, err=c.err)
        lse = lse.cpu().numpy().astype(np.float64)
        g = hq // hkv
        for b in range(2):
            n = at[b] + J
            want = np.zeros((hkv, n))
            for h in range(hkv):
                heads = slice(h * g, (h + 1) * g)
                K = keys[b][held[b][h], h:h + 1]
                given[b][h, held[b][h]] += O.attention_mass(every_q[-1][b][:, heads], K, c.desc.scale, n, lse[b][:, heads])[0]
                want[h] = given[b][h, held[b][h]]
            stacked = np.concatenate([x[b] for x in every_q])
            check_mass(mass[b, :, :n].cpu().numpy(), want, stacked, keys[b], c.desc.scale, None, (step, b))
            if step < 2:
                assert (mass[b, :, n:] == 7).all()
        if step % 3 == 2:
            keep = torch.full((2, shards), budget, dtype=torch.int32, device="cuda")
            out = dict(mass=torch.zeros_like(mass), pos=torch.zeros(mass.shape, dtype=torch.int32, device="cuda"),
                       starts=torch.zeros_like(starts), lens=torch.zeros_like(seq_lens))
            ws = torch.empty(dcp.dcp_evict_workspace_size(c.desc, 2, shards, cap), dtype=torch.uint8, device="cuda")
            before, bounds = mass.cpu(), starts.tolist()
            dcp.dcp_kv_evict(c.desc, c.shards, seq_lens, starts, keep, 2, 5, mass, out["mass"], out["pos"], out["starts"],
                             out["lens"], ws, pos_in=pos, known_lens=known, total_lens=dev(total), err=c.err)
            for b in range(2):
                for h in range(hkv):
                    kept = []
                    for i in range(shards):
                        lo, hi = O.shard_token_range(bounds[b], i, len(held[b][h]))
                        kept += (O.evict_order(before[b, h, lo:hi].tolist(), held[b][h][lo:hi], budget, 2, 5, total[b])
                                 + lo).tolist()
                    held[b][h] = [held[b][h][t] for t in kept]
                    assert out["pos"][b, h, :len(kept)].tolist() == held[b][h]
                    assert torch.equal(out["mass"][b, h, :len(kept)].cpu(), before[b, h, kept])
            starts, seq_lens, mass, pos, known = out["starts"], out["lens"], out["mass"], out["pos"], out["lens"]
    assert c.flag() == 0


@pytest.mark.parametrize("hq,hkv,d,bs", [(8, 2, 64, 16), (16, 1, 128, 32), (48, 2, 128, 16)])
def test_one_shards_range_over_the_four_bit_cache(hq, hkv, d, bs):
    """dcp_decode_partial: each shard by itself with a range of its own, open ends and empty ones among them; the merge of
    all is the whole attention."""
    lens = [300, 1, 77, 0]
    rows = normal_rows(lens, hkv, d, 83)
    c = Cache("mxfp4", lens, hq, hkv, d, bs, 3, rows)
    q = queries(4, 1, hq, d, 84).cuda()
    K, V = [as_cached("mxfp4", r[0]) for r in rows], [as_cached("mxfp4", r[1]) for r in rows]
    ws = torch.empty(dcp.dcp_workspace_size(c.desc, 4, 1), dtype=torch.uint8, device="cuda")
    o_parts, lses = torch.full((3, 4, hq, d), math.nan, device="cuda"), torch.full((3, 4, hq), math.nan, device="cuda")
    for i, shard in enumerate(c.shards):
        lo = c.starts[:, i]
        hi = c.starts[:, i + 1] if i + 1 < 3 else torch.full_like(lo, 2 ** 31 - 1)
        dcp.dcp_decode_partial(c.desc, q[:, 0].contiguous(), shard, c.seq_lens, torch.stack([lo, hi], dim=1).contiguous(),
                               o_parts[i], lses[i], ws, err=c.err)
    o, lse = torch.empty(4, hq, d, device="cuda"), torch.empty(4, hq, device="cuda")
    dcp.dcp_merge(o_parts, lses, o, lse)
    assert c.flag() == 0
    for b, n in enumerate(lens):
        qb = f64(q[b].cpu())
        for i in range(3):
            lo, hi = O.shard_token_range(c.starts_host[b].tolist(), i, n)
            ro, rl = O.attention(qb[0], K[b], V[b], c.desc.scale, lo, hi)
            check_attention(o_parts[i, b][None].cpu().numpy(), lses[i, b][None].cpu().numpy(), ro[None], rl[None], qb,
                            K[b][lo:hi], V[b][lo:hi], c.desc.scale, (b, i))
        ro, rl = O.attention(qb[0], K[b], V[b], c.desc.scale, 0, n)
        check_attention(o[b][None].cpu().numpy(), lse[b][None].cpu().numpy(), ro[None], rl[None], qb, K[b], V[b],
                        c.desc.scale, b)
