"""DecodeState through evictions: the state goes on with the next step's
tokens, loses no weight, and orders its own tensors on the caller's stream."""
import numpy as np
import pytest
import torch

import oracle as O
from compress_helpers import check_attention, check_mass
from helpers import f64
from sequence_sharded_decode_gb300 import configs, dcp
from sequence_sharded_decode_gb300.state import DecodeState

pytestmark = pytest.mark.gpu


def _state(kv, q_len=1, ctx=200, **kw):
    return DecodeState(configs.get("gqa_tiny").with_(kv_dtype=kv, batch=2, ctx_fixed=ctx, shards=2, **kw), q_len=q_len)


def _cached(st):
    """float64 (keys, values) [B][L, H, D] of every cached token, by cache index."""
    out = []
    lens = st.seq_lens.tolist()
    for b, n in enumerate(lens):
        k = torch.empty(n, st.wl.kv_heads, st.wl.dk, dtype=torch.bfloat16, device="cuda")
        v = torch.empty(n, st.wl.kv_heads, st.wl.dv, dtype=torch.bfloat16, device="cuda")
        dcp.dcp_kv_read(st.desc, st.shards, st.starts, torch.arange(n, dtype=torch.int32, device="cuda"), k, v,
                        seq_ids=torch.full((n,), b, dtype=torch.int32, device="cuda"), err=st.err)
        out.append((f64(k.cpu()), f64(v.cpu())))
    return out


def _rows_as_cached(st, k, v):
    k, v = f64(k.cpu()), f64(v.cpu())
    if st.wl.kv_dtype == "mxfp4":
        k, v = O.mx4_values(*O.mx4_quantise(k)), O.mx4_values(*O.mx4_quantise(v))
    return k, v


@pytest.mark.parametrize("kv", ["bf16", "mxfp4"])
@pytest.mark.parametrize("q_len", [1, 3])
def test_steps_after_evictions(kv, q_len):
    """step, weigh, evict, three times over: each step's tokens follow the kept ones, are attended and weighed, and every
    kept token's mass is what all steps gave it."""
    st = _state(kv, q_len)
    wl, B, hkv, g = st.wl, 2, st.wl.kv_heads, st.wl.q_heads // st.wl.kv_heads
    carried = [np.zeros((hkv, 200)) for _ in range(B)]
    pos = [np.tile(np.arange(200), (hkv, 1)) for _ in range(B)]
    total = 200
    for step, budget in enumerate((60, 40, 40)):
        st.step(fused=step != 1)
        st.weigh()
        torch.cuda.synchronize()
        assert int(st.err.item()) == 0
        n = 200 + q_len if step == 0 else len(carried[0][0]) + q_len
        total += q_len
        assert st.seq_lens.tolist() == [n, n] and st.positions.view(B, q_len).tolist() == [list(range(n - q_len, n))] * B
        want_k, want_v = _rows_as_cached(st, *st.token_rows(np.repeat(np.arange(B), q_len),
                                                            np.tile(np.arange(total - q_len, total), B)))
        cached = _cached(st)
        q = f64(st.q.cpu()).reshape(B, q_len, wl.q_heads, wl.dk)
        o, lse = st.o.cpu().numpy().reshape(B, q_len, wl.q_heads, wl.dv), st.lse.cpu().numpy().reshape(B, q_len, wl.q_heads)
        for b in range(B):
            K, V = cached[b]
            assert np.array_equal(K[n - q_len:], want_k.reshape(B, q_len, hkv, wl.dk)[b])
            assert np.array_equal(V[n - q_len:], want_v.reshape(B, q_len, hkv, wl.dv)[b])
            ro, rl = O.mtp_attention(q[b], K, V, wl.scale, n)
            check_attention(o[b], lse[b], ro, rl, q[b], K, V, wl.scale, (step, b))
            w = O.attention_mass(q[b], K, wl.scale, n, lse[b].astype(np.float64))
            carried[b] = np.concatenate([carried[b], np.zeros((hkv, q_len))], axis=1) + w
            pos[b] = np.concatenate([pos[b], np.tile(np.arange(total - q_len, total), (hkv, 1))], axis=1)
            got = st.mass[b, :, :n].cpu().numpy()
            # every step's weight within its own bound: their errors add up
            check_mass(got, carried[b], np.concatenate([q[b]] * (step + 1)), K, wl.scale, None, (step, b))
        before = st.mass.cpu()
        starts = st.starts.tolist()
        st.evict(torch.full((B, 2), budget, dtype=torch.int32, device="cuda"), n_sink=2, n_recent=20)
        torch.cuda.synchronize()
        assert int(st.err.item()) == 0 and st.seq_lens.tolist() == [2 * budget] * B
        for b in range(B):
            keep_m, keep_p = [], []
            for h in range(hkv):
                order = []
                for i in range(2):
                    lo, hi = O.shard_token_range(starts[b], i, n)
                    order += (O.evict_order(before[b, h, lo:hi].tolist(), pos[b][h, lo:hi].tolist(), budget, 2, 20, total)
                              + lo).tolist()
                keep_m.append(carried[b][h, order])
                keep_p.append(pos[b][h, order])
                assert st.pos[b, h, :2 * budget].tolist() == keep_p[-1].tolist()
                assert torch.equal(st.mass[b, h, :2 * budget].cpu(), before[b, h, order])
            carried[b], pos[b] = np.stack(keep_m), np.stack(keep_p)
    assert st.attended_tokens() == B * 80 and st.kv_bytes() == B * 80 * wl.kv_bytes_per_token


def test_weighing_the_kept_tokens_again_loses_nothing():
    """A step of one token may attend and weigh what an eviction left, before the next token comes: all masses grow."""
    st = _state("mxfp4")
    st.step(fused=True)
    st.weigh()
    st.evict(torch.full((2, 2), 40, dtype=torch.int32, device="cuda"))
    before = st.mass[:, :, :80].clone()
    st.attention()
    st.weigh()
    grown = (st.mass[:, :, :80] - before).double()
    assert (grown >= 0).all() and torch.allclose(grown.sum(-1), torch.full((2, 2), 4.0, device="cuda", dtype=torch.float64),
                                                 atol=1e-3)
    assert (st.mass[:, :, 80:] == 0).all() and int(st.err.item()) == 0


def test_several_query_tokens_wait_for_their_own():
    """Attention of several query tokens is causal among the last cached tokens, which after an eviction are any."""
    st = _state("bf16", q_len=2)
    st.step(fused=True)
    st.weigh()
    st.evict(torch.full((2, 2), 40, dtype=torch.int32, device="cuda"))
    for call in (st.attention, st.partial, st.weigh):
        with pytest.raises(RuntimeError, match="append"):
            call()
    st.append()
    st.attention()
    st.weigh()
    torch.cuda.synchronize()
    assert st.seq_lens.tolist() == [82, 82] and int(st.err.item()) == 0


def test_evictions_in_a_row():
    st = _state("bf16")
    st.step(fused=True)
    st.weigh()
    for budget in (50, 30, 20, 10):
        before, pos = st.mass.clone(), None if st.pos is None else st.pos.clone()
        n = st.seq_lens.tolist()[0]
        st.evict(torch.full((2, 2), budget, dtype=torch.int32, device="cuda"), n_sink=0, n_recent=0)
        torch.cuda.synchronize()
        assert st.seq_lens.tolist() == [2 * budget] * 2
        for h in range(2):  # the heaviest of either shard
            kept = torch.cat([torch.sort(before[0, h, a:e], descending=True)[0][:budget]
                              for a, e in ((0, n // 2 if pos is not None else 100), (n // 2 if pos is not None else 100, n))])
            assert torch.equal(torch.sort(st.mass[0, h, :2 * budget])[0], torch.sort(kept)[0])
    st.step(fused=True)
    torch.cuda.synchronize()
    assert st.seq_lens.tolist() == [21, 21] and int(st.err.item()) == 0


def test_calls_on_a_stream_of_their_own():
    """Work on the current stream is not waited for and does not reach into the calls on another one."""
    keep = torch.full((2, 2), 40, dtype=torch.int32, device="cuda")
    want = _state("bf16")
    want.step(fused=True)
    want.weigh()
    want.evict(keep)
    want.step(fused=True)
    want.weigh()
    torch.cuda.synchronize()
    st = _state("bf16")
    st.step(fused=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(100_000_000)                        # ~50 ms, on the current stream
    st.weigh(stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    st.evict(keep, stream=side.cuda_stream)
    st.step(stream=side, fused=True)
    st.weigh(stream=side.cuda_stream)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(st.seq_lens, want.seq_lens) and torch.equal(st.pos[:, :, :80], want.pos[:, :, :80])
    assert torch.equal(st.mass[:, :, :81], want.mass[:, :, :81]) and torch.equal(st.o, want.o)
    assert int(st.err.item()) == 0


def test_memory_let_go_is_not_reused_under_a_waiting_call():
    """Tensors that an eviction on a busy stream replaces stay as they are until it has run, whatever the current stream
    allocates meanwhile."""
    keep = torch.full((2, 2), 40, dtype=torch.int32, device="cuda")
    results = []
    for wait in (False, True):
        st = _state("bf16", ctx=2000)
        st.step(fused=True)
        st.weigh()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            if wait:
                torch.cuda._sleep(200_000_000)            # ~100 ms
        sizes = [st.mass.numel(), st.starts.numel(), st.seq_lens.numel()]
        st.evict(keep, stream=side)
        st.step(stream=side, fused=True)
        junk = [torch.full((n,), 3, dtype=torch.int32, device="cuda") for n in sizes * 20]  # on the current stream
        torch.cuda.synchronize()
        results.append((st.mass[:, :, :80].clone(), st.pos[:, :, :80].clone(), st.o.clone()))
        assert int(st.err.item()) == 0 and len(junk) == 60
    assert all(torch.equal(a, b) for a, b in zip(*results))
