"""Device state of one decode step for a workload preset.

Allocates the N shard pools, block tables, queries, the step's new tokens,
the reused workspace and the output buffers with torch, fills the pools
through dcp_kv_append, and runs one step through the C ABI:
append -> partial attention on every shard -> LSE merge. weigh() and evict()
add the eviction of the cached tokens with the least attention weight.
"""
from __future__ import annotations

import contextlib

import numpy as np
import torch

from . import configs, dcp, inputs


def _on(stream):
    """Context in which torch's own work and memory belong to `stream` (a
    torch stream, a handle, or None for the current one)."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream)) if stream else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _release(*tensors):
    """Before tensors are dropped: their memory, of whichever stream, is kept
    until the current stream has run what reads them."""
    for t in tensors:
        if t is not None:
            t.record_stream(torch.cuda.current_stream())


class DecodeState:
    def __init__(self, wl: configs.Workload, device: str = "cuda", fill: bool = True,
                 canary: int | None = None, table_seed: int | None = None, fill_chunk: int = 1 << 18,
                 q_len: int = 1, gen_device: str | None = None):
        """q_len > 1: every sequence brings q_len new tokens per step (a
        speculative / multi-token step); query token j sits at position
        ctx[b] + j and the partial pass is dcp_decode_partial_all_mtp.
        gen_device: where the seeded draws are made before they are copied to
        `device` (default: on `device`; "cpu" for small cases keeps the
        device's launch list to the library's own kernels)."""
        self.wl = wl
        self.device = device
        self.gen = device if gen_device is None else gen_device
        self.q_len = q_len
        self.ctx = wl.ctx_lens().astype(np.int64)
        B, N = wl.batch, wl.shards
        self.f8 = wl.kv_dtype == "fp8"
        kv = {"bf16": dcp.DCP_KV_BF16, "fp8": dcp.DCP_KV_FP8_E4M3, "mxfp4": dcp.DCP_KV_MXFP4}[wl.kv_dtype]
        self.desc = dcp.AttnDesc(wl.kind, wl.q_heads, wl.kv_heads, wl.dk, wl.dv, wl.block_size, wl.scale, kv,
                                 wl.k_scale, wl.v_scale)
        starts, blocks = dcp.dcp_shard_plan(self.ctx, N, wl.block_size, q_len)
        self.starts_host, self.blocks_host = starts, blocks
        seed_t = wl.seed + 1 if table_seed is None else table_seed
        self.tables_host = inputs.block_tables(seed_t, blocks, wl.capacity_factor)
        self.shards = []
        for cap, tab in self.tables_host:
            # MLA: one latent row per token and no values; E4M3 values and 4-bit tiles have layouts of their own
            ks, vs = self.desc.pool_shapes(cap)
            k = torch.empty(ks, dtype=self.desc.kv_torch_dtype, device=device)
            v = None if vs is None else torch.empty(vs, dtype=self.desc.kv_torch_dtype, device=device)
            if canary is not None:
                for pool in (k, v):
                    if pool is None:
                        continue
                    if pool.dtype == torch.uint8:
                        pool.fill_(canary & 0xFF)
                    else:
                        pool.view(torch.int16).fill_(canary)
            self.shards.append(dcp.Shard(k, v, torch.from_numpy(tab).to(device)))
        self.starts = torch.from_numpy(starts).to(device)
        qstream = inputs.STREAM_Q_MLA if wl.kind == configs.MLA else inputs.STREAM_Q
        if q_len == 1:
            self.q = inputs.query(wl.seed, np.arange(B), wl.q_heads, wl.dk, self.gen, stream=qstream).to(device)
            self.q0 = self.q
        else:
            self.q = inputs.query_tokens(wl.seed, np.arange(B), q_len, wl.q_heads, wl.dk, self.gen,
                                         stream=qstream).to(device)
            self.q0 = self.q[:, 0].contiguous()  # planted needles copy query token 0
        self.needles = wl.needle_plan()
        new_b = np.repeat(np.arange(B), q_len)
        new_t = (self.ctx[:, None] + np.arange(q_len)[None, :]).reshape(-1)
        self.seq_ids = torch.from_numpy(new_b.astype(np.int32)).to(device) if q_len > 1 else None
        self.positions = torch.from_numpy(new_t.astype(np.int32)).to(device)
        self.seq_lens = torch.from_numpy((self.ctx + q_len).astype(np.int32)).to(device)
        self.k_new, self.v_new = self.token_rows(new_b, new_t)
        ws = dcp.dcp_workspace_size_mtp(self.desc, B, q_len, N)
        if ws <= 0:
            raise RuntimeError("dcp_workspace_size failed")
        self.workspace = torch.empty(ws, dtype=torch.uint8, device=device)
        rows = (B,) if q_len == 1 else (B, q_len)
        self.o_parts = torch.empty((N, *rows, wl.q_heads, wl.dv), dtype=torch.float32, device=device)
        self.lses = torch.empty((N, *rows, wl.q_heads), dtype=torch.float32, device=device)
        self.o = torch.empty((*rows, wl.q_heads, wl.dv), dtype=torch.float32, device=device)
        self.lse = torch.empty((*rows, wl.q_heads), dtype=torch.float32, device=device)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)
        self.steps_taken = 0        # after the first one
        self.between_steps = False  # after an eviction, until the next step's tokens are appended
        if fill:
            self.fill_context(fill_chunk)

    # -- token rows from the seeded generator -------------------------------
    def token_rows(self, b, t):
        """K/V (or latent) rows of tokens (b[j], t[j]), drawn on the generation
        device and returned on the state's device."""
        wl = self.wl
        g = self.gen
        b = torch.as_tensor(b).to(g)
        t = torch.as_tensor(t).to(g)
        if wl.kind == configs.MLA:
            lat = inputs.kv_tokens(wl.seed, inputs.STREAM_LATENT, b, t, 1, wl.dk, g, chunk=1 << 18)
            lat = inputs.plant_needles(lat.view(-1, wl.dk), b, t, self.q0.to(g), self.needles, wl.q_heads)
            if self.f8:  # the cache holds the E4M3 codes of the same draws
                lat = inputs.e4m3_codes(lat)
            return lat.to(self.device), None
        k = inputs.kv_tokens(wl.seed, inputs.STREAM_K, b, t, wl.kv_heads, wl.dk, g, chunk=1 << 16)
        k = inputs.plant_needles(k, b, t, self.q0.to(g), self.needles, wl.q_heads)
        v = inputs.kv_tokens(wl.seed, inputs.STREAM_V, b, t, wl.kv_heads, wl.dv, g, chunk=1 << 16)
        if self.f8:  # the cache holds the E4M3 codes of the same draws
            k, v = inputs.e4m3_codes(k), inputs.e4m3_codes(v)
        return k.to(self.device), v.to(self.device)

    def fill_context(self, chunk: int = 1 << 18):
        """Write every context token [0, ctx[b]) of every sequence into the pools."""
        ctx = torch.from_numpy(self.ctx).to(self.gen)
        ends = torch.cumsum(ctx, 0)
        begins = ends - ctx
        total = int(ends[-1]) if ctx.numel() else 0
        for s in range(0, total, chunk):
            idx = torch.arange(s, min(total, s + chunk), dtype=torch.int64, device=self.gen)
            b = torch.searchsorted(ends, idx, right=True)
            t = idx - begins[b]
            k, v = self.token_rows(b, t)
            dcp.dcp_kv_append(self.desc, self.shards, self.starts, t.to(torch.int32).to(self.device), k, v,
                              seq_ids=b.to(torch.int32).to(self.device), err=self.err)

    # -- the decode step through the C ABI ------------------------------------
    def append(self, stream=None):
        """The step's tokens into the cache; after an eviction those of the next
        step (advance())."""
        if self.between_steps:
            self.advance(stream)
        dcp.dcp_kv_append(self.desc, self.shards, self.starts, self.positions, self.k_new, self.v_new,
                          seq_ids=self.seq_ids, err=self.err, stream=stream)

    def _check_appended(self):
        # several query tokens see each other causally, as the last q_len cached tokens
        if self.between_steps and self.q_len > 1:
            raise RuntimeError("after an eviction, append the next step's tokens first")

    def partial(self, stream=None):
        self._check_appended()
        if self.q_len == 1:
            dcp.dcp_decode_partial_all(self.desc, self.q, self.shards, self.seq_lens, self.starts, self.o_parts,
                                       self.lses, self.workspace, err=self.err, stream=stream)
        else:
            dcp.dcp_decode_partial_all_mtp(self.desc, self.q, self.shards, self.seq_lens, self.starts,
                                           self.o_parts, self.lses, self.workspace, err=self.err, stream=stream)

    def attention(self, stream=None):
        """Partial attention of every shard and the merge in one call."""
        self._check_appended()
        dcp.dcp_attention_all(self.desc, self.q, self.shards, self.seq_lens, self.starts, self.o_parts, self.lses,
                              self.o, self.lse, self.workspace, err=self.err, stream=stream)

    def merge(self, stream=None):
        dcp.dcp_merge(self.o_parts, self.lses, self.o, self.lse, stream=stream)

    # -- eviction ---------------------------------------------------------------
    def weigh(self, stream=None):
        """Add the attention weight that this step gave every cached token (after
        attention() or partial() and merge(), whose LSE it takes)."""
        self._check_appended()
        with _on(stream):
            if not hasattr(self, "mass"):
                cap = int(self.ctx.max()) + self.q_len if self.wl.batch else 1
                self.mass = torch.zeros((self.wl.batch, self.wl.kv_heads, cap), dtype=torch.float32, device=self.device)
                self.pos = self.known_lens = None
                self.total_lens = self.seq_lens.clone()
            # right after an eviction none of the cached tokens is the step's own, whose weight would start at 0
            here = torch.zeros_like(self.mass) if self.between_steps else self.mass
            dcp.dcp_attention_mass(self.desc, self.q, self.shards, self.seq_lens, self.starts, self.lse, here,
                                   mass_in=None if self.between_steps else here, err=self.err)
            if self.between_steps:
                self.mass += here

    def evict(self, keep: torch.Tensor, n_sink: int = 4, n_recent: int = 32, stream=None):
        """Keep the keep[b, i] (int32 [B, N]) heaviest tokens of every shard and
        KV head. The state goes on with the shortened sequences: the next
        append() brings the next step's tokens. (A state of one query token may
        attend and weigh the kept ones again before that.)"""
        wl = self.wl
        cap = self.mass.shape[-1]
        with _on(stream):
            if not hasattr(self, "evict_workspace"):
                size = dcp.dcp_evict_workspace_size(self.desc, wl.batch, wl.shards, cap)
                self.evict_workspace = torch.empty(size, dtype=torch.uint8, device=self.device)
            mass, pos = torch.zeros_like(self.mass), torch.zeros(self.mass.shape, dtype=torch.int32, device=self.device)
            starts, lens = torch.empty_like(self.starts), torch.empty_like(self.seq_lens)
            dcp.dcp_kv_evict(self.desc, self.shards, self.seq_lens, self.starts, keep, n_sink, n_recent, self.mass,
                             mass, pos, starts, lens, self.evict_workspace, pos_in=self.pos,
                             known_lens=self.known_lens, total_lens=self.total_lens, err=self.err)
            _release(keep, self.mass, self.pos, self.starts, self.seq_lens, self.known_lens)
        self.mass, self.pos, self.starts, self.seq_lens, self.known_lens = mass, pos, starts, lens, lens
        self.between_steps = True

    def advance(self, stream=None):
        """On to the next step after an eviction (append() does it): its tokens
        follow the kept ones in the cache, at index seq_lens of the last shard,
        whose freed blocks take them, and the evicted ones too in the text, where
        total_lens counts. One that finds no room raises the error flag."""
        if not self.between_steps:
            raise RuntimeError("the step's tokens are the state's last ones already")
        B, J = self.wl.batch, self.q_len
        text = (self.ctx + J * (self.steps_taken + 1)).repeat(J) + np.tile(np.arange(J), B)
        with _on(stream):
            k, v = self.token_rows(np.repeat(np.arange(B), J), text)
            _release(self.k_new, self.v_new, self.positions, self.seq_lens, self.total_lens)
            self.k_new, self.v_new = k, v
            new = torch.arange(J, dtype=torch.int32, device=self.device)
            self.positions = (self.known_lens[:, None] + new).reshape(-1)
            self.seq_lens = self.known_lens + J
            self.total_lens = self.total_lens + J
        self.steps_taken += 1
        self.between_steps = False

    def step(self, stream=None, fused: bool = False):
        """append -> partial attention of every shard -> merge; fused: the last
        two in one call (dcp_attention_all; the shards' partial rows of split
        ranges -- for MLA, all of them -- are then not written), else
        dcp_decode_partial_all(_mtp) then dcp_merge."""
        self.append(stream)
        if fused:
            self.attention(stream)
        else:
            self.partial(stream)
            self.merge(stream)

    # -- algorithmic bytes ---------------------------------------------------
    def _cached(self) -> np.ndarray:
        """Tokens cached before the step, per sequence (after an eviction they are
        read from the device)."""
        if not self.steps_taken and not self.between_steps:
            return self.ctx
        return self.seq_lens.cpu().numpy().astype(np.int64) - self.q_len

    def attended_tokens(self) -> int:
        """Distinct tokens the step attends: the context plus the new tokens
        (with several query tokens, each token is still read from HBM once)."""
        return int((self._cached() + self.q_len).sum())

    def attention_flops(self) -> int:
        """Multiply-add flops of the partial pass: for every query token, q.k
        and p.v over each token it attends (2 (Dk + Dv) per head and token)."""
        wl = self.wl
        per_seq = self.q_len * (self._cached() + 1) + self.q_len * (self.q_len - 1) // 2  # sum_j (ctx + j + 1)
        return int(2 * wl.q_heads * (wl.dk + wl.dv) * per_seq.sum())

    def kv_bytes(self) -> int:
        """KV bytes the partial-attention pass must read (each attended token once)."""
        return self.attended_tokens() * self.wl.kv_bytes_per_token

    def step_bytes(self, fused: bool = False) -> dict:
        """Algorithmic HBM bytes of one step, by call. Two calls (and GQA's
        one call): the shards' partial rows are written and read back. MLA's
        one call merges the shards on chip: KV, queries and the merged rows
        only (the pieces of the few row groups a CTA boundary cuts are left
        out: at most two per CTA pair)."""
        wl = self.wl
        B, N, Hq, dv, dk = wl.batch * self.q_len, wl.shards, wl.q_heads, wl.dv, wl.dk
        part = N * B * Hq * (dv + 1) * 4
        out = B * Hq * (dv + 1) * 4
        new_tok = B * (wl.kv_bytes_per_token if wl.kind == configs.GQA else dk * 2)
        rows_in = B * 2 * wl.kv_heads * (dk + dv) if wl.kv_dtype == "mxfp4" else new_tok  # quantised from bf16
        if fused and wl.kind == configs.MLA:
            return {
                "append": rows_in + new_tok,            # read the new rows, write them
                "attention": self.kv_bytes() + B * Hq * dk * 2 + out,
            }
        return {
            "append": rows_in + new_tok,
            "partial": self.kv_bytes() + B * Hq * dk * 2 + part,
            "merge": part + out,
        }
