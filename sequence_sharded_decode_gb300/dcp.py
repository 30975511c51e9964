"""Python binding of libdcp's C ABI (argument marshalling only).

Every function here has the name of the C entry point it calls and does no
arithmetic of its own: it checks dtypes/devices/contiguity, turns torch
tensors into raw pointers and passes them on. There is no fallback: if the
compiled library is missing the import of this module's functions raises.
"""
from __future__ import annotations

import ctypes
import functools
import operator
import os
from dataclasses import dataclass

import numpy as np
import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdcp.so")
_lib = None

DCP_OK = 0
DCP_ERR_INVALID_ARG = -1
DCP_ERR_SHAPE = -2
DCP_ERR_UNSUPPORTED = -3
DCP_ERR_CUDA = -4
DCP_ERR_WORKSPACE = -5
DCP_ERR_SCRATCH_LIMIT = -6
DCP_NOALLOC_SCRATCH_BYTES = 64 << 20

DCP_DEVERR_BLOCK_RANGE = 1
DCP_DEVERR_TABLE_RANGE = 2
DCP_DEVERR_POSITION = 4
DCP_DEVERR_TIMEOUT = 8
DCP_DEVERR_NONFINITE = 16

DCP_MAX_SHARDS = 32
DCP_MAX_QUERY_TOKENS = 8192
DCP_KIND_GQA = 0
DCP_KIND_MLA = 1
DCP_KV_BF16 = 0
DCP_KV_FP8_E4M3 = 1
DCP_KV_MXFP4 = 4

EXPORTED = ("dcp_status_string", "dcp_version", "dcp_shard_plan", "dcp_kv_append", "dcp_workspace_size",
            "dcp_workspace_size_mtp", "dcp_decode_partial", "dcp_decode_partial_all", "dcp_decode_partial_all_mtp",
            "dcp_attention_all",
            "dcp_decode_partial_all_noalloc", "dcp_merge", "dcp_kv_read", "dcp_attention_mass",
            "dcp_evict_workspace_size", "dcp_kv_evict")


class DcpError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {dcp_status_string(status)} ({status})")
        self.status = status


class _Desc(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("num_q_heads", ctypes.c_int), ("num_kv_heads", ctypes.c_int),
                ("head_dim_k", ctypes.c_int), ("head_dim_v", ctypes.c_int), ("block_size", ctypes.c_int),
                ("scale", ctypes.c_float), ("kv_dtype", ctypes.c_int), ("k_scale", ctypes.c_float),
                ("v_scale", ctypes.c_float)]


class _Shard(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p), ("num_blocks", ctypes.c_int64),
                ("block_table", ctypes.c_void_p), ("max_blocks_per_seq", ctypes.c_int32)]


@dataclass(frozen=True)
class AttnDesc:
    kind: int
    num_q_heads: int
    num_kv_heads: int
    head_dim_k: int
    head_dim_v: int
    block_size: int
    scale: float
    kv_dtype: int = DCP_KV_BF16
    k_scale: float = 1.0
    v_scale: float = 1.0

    def c(self) -> _Desc:
        """The descriptor's library form, the caller's own."""
        return _Desc.from_buffer_copy(self._c)

    @functools.cached_property
    def _c(self) -> _Desc:  # the calls' (the fields are frozen, and the library only reads it)
        return _Desc(self.kind, self.num_q_heads, self.num_kv_heads, self.head_dim_k, self.head_dim_v,
                     self.block_size, self.scale, self.kv_dtype, self.k_scale, self.v_scale)

    @functools.cached_property
    def kv_torch_dtype(self):
        """torch dtype of the pools: bf16, or uint8 codes (E4M3, or 4-bit tiles)."""
        return torch.bfloat16 if self.kv_dtype == DCP_KV_BF16 else torch.uint8

    @functools.cached_property
    def row_torch_dtype(self):
        """torch dtype of appended rows: bf16, or uint8 E4M3 codes."""
        return torch.uint8 if self.kv_dtype == DCP_KV_FP8_E4M3 else torch.bfloat16

    @functools.cached_property
    def block_shapes(self):
        """Shapes of a block in the key and the value pool (None for MLA's values)."""
        h, bs, dk, dv = self.num_kv_heads, self.block_size, self.head_dim_k, self.head_dim_v
        if self.kind == DCP_KIND_MLA:
            return (bs, dk), None
        if self.kv_dtype == DCP_KV_MXFP4:
            return (h, bs * (dk // 2 + dk // 32)), (h, bs * (dv // 2 + dv // 32))
        return (h, bs, dk), ((h, dv, bs) if self.kv_dtype == DCP_KV_FP8_E4M3 else (h, bs, dv))

    def pool_shapes(self, num_blocks: int):
        """Shapes of a shard's key and value pools (None for MLA's values)."""
        k, v = self.block_shapes
        return (num_blocks, *k), None if v is None else (num_blocks, *v)


@dataclass
class Shard:
    """One shard's pool(s) and block table (device tensors).

    The tensors are checked and their library form is made when the shard is
    first used, and again after a field is set or a tensor's storage, shape,
    type or order changes."""
    k_pool: torch.Tensor
    v_pool: torch.Tensor | None
    block_table: torch.Tensor

    def __setattr__(self, name, value):
        self.__dict__[name] = value
        self.__dict__["_made"] = None

    def __getstate__(self):
        return {"k_pool": self.k_pool, "v_pool": self.v_pool, "block_table": self.block_table}

    def __setstate__(self, state):
        for name, value in state.items():
            setattr(self, name, value)

    def c(self) -> _Shard:
        """The shard's library form, the caller's own."""
        return _Shard.from_buffer_copy(self._form()[0])

    def _form(self):
        """(library form, what it was made of, (device, pool type, table rows, elements of a key and a value block))"""
        made, k, v, t = self._made, self.k_pool, self.v_pool, self.block_table
        # (strides and bytes stand for the shape, which takes longer to ask for)
        if v is None:
            now = (k.data_ptr(), t.data_ptr(), k.stride(), t.stride(), k.nbytes, t.nbytes, k.dtype, t.dtype)
        else:
            now = (k.data_ptr(), t.data_ptr(), k.stride(), t.stride(), k.nbytes, t.nbytes, k.dtype, t.dtype, v.data_ptr(),
                   v.stride(), v.nbytes, v.dtype)
        if made is not None and made[1] == now:
            return made
        if k.dtype not in (torch.bfloat16, torch.uint8):
            raise TypeError("k_pool must be bf16 or uint8 (E4M3 codes, 4-bit tiles)")
        _check(k, k.dtype, "k_pool")
        if v is not None:
            _check(v, k.dtype, "v_pool")
        _check(t, torch.int32, "block_table")
        devices = {x.device for x in (k, v, t) if x is not None}
        what = (devices.pop() if len(devices) == 1 else None, k.dtype, int(t.shape[0]) if t.dim() == 2 else -1,
                tuple(k.shape[1:]), None if v is None else tuple(v.shape[1:]))
        made = (_Shard(now[0], None if v is None else now[8], int(k.shape[0]), now[1], int(t.shape[1])), now, what)
        self.__dict__["_made"] = made
        return made


def lib_path() -> str:
    return _LIB_PATH


def load() -> ctypes.CDLL:
    """Load libdcp.so (built in-tree by build.py); raises if it is absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"libdcp.so not built ({_LIB_PATH}); run sequence_sharded_decode_gb300.build.build()")
    lib = ctypes.CDLL(_LIB_PATH)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    pdesc, pshard = ctypes.POINTER(_Desc), ctypes.POINTER(_Shard)
    lib.dcp_status_string.restype = ctypes.c_char_p
    lib.dcp_status_string.argtypes = [i32]
    lib.dcp_version.restype = i32
    lib.dcp_version.argtypes = []
    lib.dcp_shard_plan.restype = i32
    lib.dcp_shard_plan.argtypes = [vp, i32, i32, i32, i32, vp, vp]
    lib.dcp_kv_append.restype = i32
    lib.dcp_kv_append.argtypes = [pdesc, pshard, i32, vp, i32, vp, vp, vp, vp, i32, vp, vp]
    lib.dcp_workspace_size.restype = sz
    lib.dcp_workspace_size.argtypes = [pdesc, i32, i32]
    lib.dcp_workspace_size_mtp.restype = sz
    lib.dcp_workspace_size_mtp.argtypes = [pdesc, i32, i32, i32]
    lib.dcp_decode_partial.restype = i32
    lib.dcp_decode_partial.argtypes = [pdesc, vp, pshard, vp, vp, i32, vp, vp, vp, sz, vp, vp]
    lib.dcp_decode_partial_all.restype = i32
    lib.dcp_decode_partial_all.argtypes = [pdesc, vp, pshard, i32, vp, vp, i32, vp, vp, vp, sz, vp, vp]
    lib.dcp_decode_partial_all_mtp.restype = i32
    lib.dcp_decode_partial_all_mtp.argtypes = [pdesc, vp, pshard, i32, vp, vp, i32, i32, vp, vp, vp, sz, vp, vp]
    lib.dcp_attention_all.restype = i32
    lib.dcp_attention_all.argtypes = [pdesc, vp, pshard, i32, vp, vp, i32, i32, vp, vp, vp, vp, vp, sz, vp, vp]
    lib.dcp_decode_partial_all_noalloc.restype = i32
    lib.dcp_decode_partial_all_noalloc.argtypes = [pdesc, vp, pshard, i32, vp, vp, i32, vp, vp, vp, vp]
    lib.dcp_merge.restype = i32
    lib.dcp_merge.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp]
    i64 = ctypes.c_int64
    lib.dcp_kv_read.restype = i32
    lib.dcp_kv_read.argtypes = [pdesc, pshard, i32, vp, i32, vp, vp, vp, vp, i32, vp, vp]
    lib.dcp_attention_mass.restype = i32
    lib.dcp_attention_mass.argtypes = [pdesc, vp, pshard, i32, vp, vp, i32, i32, vp, vp, vp, i64, vp, vp]
    lib.dcp_evict_workspace_size.restype = sz
    lib.dcp_evict_workspace_size.argtypes = [pdesc, i32, i32, i64]
    lib.dcp_kv_evict.restype = i32
    lib.dcp_kv_evict.argtypes = [pdesc, pshard, i32, vp, vp, i32, vp, i32, i32, vp, vp, vp, vp, i64, vp, vp, vp, vp,
                                 vp, sz, vp, vp]
    _lib = lib
    return lib


def _check(t: torch.Tensor, dtype, name: str, cuda: bool = True):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if cuda and not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")


def _ptr(t):
    return None if t is None else t.data_ptr()


# the current stream's handle without making a torch.cuda.Stream (3 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# the current device without looking whether CUDA is up (the tensors are there)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream) -> int | None:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(_current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


_SHARD_ARRAYS = [_Shard * n for n in range(DCP_MAX_SHARDS + 1)]


def _shards(shards) -> ctypes.Array:
    return _array(shards, [s._form() for s in shards])


def _array(shards, forms) -> ctypes.Array:
    """The library forms side by side: those of the last call, kept with the
    first shard, if they are the same."""
    n = len(forms)
    if n == 0:
        return _SHARD_ARRAYS[0]()
    kept = shards[0].__dict__.get("_array")
    if kept is not None and len(kept[0]) == n and all(map(operator.is_, kept[0], forms)):
        return kept[1]
    arr = (_SHARD_ARRAYS[n] if n <= DCP_MAX_SHARDS else _Shard * n)()
    for i, form in enumerate(forms):
        arr[i] = form[0]
    shards[0].__dict__["_array"] = (forms, arr)
    return arr


def _raise(rc: int, where: str):
    if rc != DCP_OK:
        raise DcpError(rc, where)


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------
def dcp_status_string(status: int) -> str:
    return load().dcp_status_string(int(status)).decode()


def dcp_version() -> int:
    return load().dcp_version()


def dcp_shard_plan(ctx_lens, n_shards: int, block_size: int, reserve_tokens: int):
    """Host routing plan: (shard_starts int32 [B, N], blocks_needed int32 [B, N])."""
    ctx = np.ascontiguousarray(np.asarray(ctx_lens, dtype=np.int32).reshape(-1))
    B = ctx.shape[0]
    starts = np.zeros((B, n_shards), dtype=np.int32)
    blocks = np.zeros((B, n_shards), dtype=np.int32)
    rc = load().dcp_shard_plan(ctx.ctypes.data, B, n_shards, block_size, reserve_tokens,
                               starts.ctypes.data, blocks.ctypes.data)
    _raise(rc, "dcp_shard_plan")
    return starts, blocks


def dcp_kv_append(desc: AttnDesc, shards, shard_starts: torch.Tensor, positions: torch.Tensor,
                  k_new: torch.Tensor, v_new: torch.Tensor | None, seq_ids: torch.Tensor | None = None,
                  err: torch.Tensor | None = None, stream=None):
    _check(shard_starts, torch.int32, "shard_starts")
    _check(positions, torch.int32, "positions")
    _check(k_new, desc.row_torch_dtype, "k_new")
    if v_new is not None:
        _check(v_new, desc.row_torch_dtype, "v_new")
    if seq_ids is not None:
        _check(seq_ids, torch.int32, "seq_ids")
    if err is not None:
        _check(err, torch.int32, "err")
    B = int(shard_starts.shape[0])
    T = int(positions.numel())
    arr = _shards(shards)
    rc = load().dcp_kv_append(ctypes.byref(desc._c), arr, len(shards), shard_starts.data_ptr(), B,
                              _ptr(seq_ids), positions.data_ptr(), k_new.data_ptr(), _ptr(v_new), T,
                              _ptr(err), _stream(stream))
    _raise(rc, "dcp_kv_append")


def dcp_workspace_size(desc: AttnDesc, batch: int, n_shards: int) -> int:
    return int(load().dcp_workspace_size(ctypes.byref(desc._c), batch, n_shards))


def dcp_workspace_size_mtp(desc: AttnDesc, batch: int, q_len: int, n_shards: int) -> int:
    return int(load().dcp_workspace_size_mtp(ctypes.byref(desc._c), batch, q_len, n_shards))


def dcp_decode_partial(desc: AttnDesc, q: torch.Tensor, shard: Shard, seq_lens: torch.Tensor,
                       shard_range: torch.Tensor, o_part: torch.Tensor, lse: torch.Tensor,
                       workspace: torch.Tensor, err: torch.Tensor | None = None, stream=None):
    _check(q, torch.bfloat16, "q")
    _check(seq_lens, torch.int32, "seq_lens")
    _check(shard_range, torch.int32, "shard_range")
    _check(o_part, torch.float32, "o_part")
    _check(lse, torch.float32, "lse")
    _check(workspace, torch.uint8, "workspace")
    if err is not None:
        _check(err, torch.int32, "err")
    arr = _shards([shard])
    rc = load().dcp_decode_partial(ctypes.byref(desc._c), q.data_ptr(), arr, seq_lens.data_ptr(),
                                   shard_range.data_ptr(), int(q.shape[0]), o_part.data_ptr(), lse.data_ptr(),
                                   workspace.data_ptr(), workspace.numel(), _ptr(err), _stream(stream))
    _raise(rc, "dcp_decode_partial")


def dcp_decode_partial_all(desc: AttnDesc, q: torch.Tensor, shards, seq_lens: torch.Tensor,
                           shard_starts: torch.Tensor, o_parts: torch.Tensor, lses: torch.Tensor,
                           workspace: torch.Tensor, err: torch.Tensor | None = None, stream=None):
    _check(q, torch.bfloat16, "q")
    _check(seq_lens, torch.int32, "seq_lens")
    _check(shard_starts, torch.int32, "shard_starts")
    _check(o_parts, torch.float32, "o_parts")
    _check(lses, torch.float32, "lses")
    _check(workspace, torch.uint8, "workspace")
    if err is not None:
        _check(err, torch.int32, "err")
    arr = _shards(shards)
    rc = load().dcp_decode_partial_all(ctypes.byref(desc._c), q.data_ptr(), arr, len(shards),
                                       seq_lens.data_ptr(), shard_starts.data_ptr(), int(q.shape[0]),
                                       o_parts.data_ptr(), lses.data_ptr(), workspace.data_ptr(),
                                       workspace.numel(), _ptr(err), _stream(stream))
    _raise(rc, "dcp_decode_partial_all")


def dcp_decode_partial_all_mtp(desc: AttnDesc, q: torch.Tensor, shards, seq_lens: torch.Tensor,
                               shard_starts: torch.Tensor, o_parts: torch.Tensor, lses: torch.Tensor,
                               workspace: torch.Tensor, err: torch.Tensor | None = None, stream=None):
    """q [B, q_len, Hq, Dk] bf16: q_len new tokens per sequence, query token j
    at position seq_lens[b] - q_len + j, causal among the new tokens.
    o_parts [N, B, q_len, Hq, Dv], lses [N, B, q_len, Hq]; the workspace is
    dcp_workspace_size_mtp(desc, B, q_len, N) bytes."""
    _check(q, torch.bfloat16, "q")
    _check(seq_lens, torch.int32, "seq_lens")
    _check(shard_starts, torch.int32, "shard_starts")
    _check(o_parts, torch.float32, "o_parts")
    _check(lses, torch.float32, "lses")
    _check(workspace, torch.uint8, "workspace")
    if err is not None:
        _check(err, torch.int32, "err")
    if q.dim() != 4:
        raise ValueError("q must be [B, q_len, Hq, Dk]")
    arr = _shards(shards)
    rc = load().dcp_decode_partial_all_mtp(ctypes.byref(desc._c), q.data_ptr(), arr, len(shards),
                                           seq_lens.data_ptr(), shard_starts.data_ptr(), int(q.shape[0]),
                                           int(q.shape[1]), o_parts.data_ptr(), lses.data_ptr(),
                                           workspace.data_ptr(), workspace.numel(), _ptr(err), _stream(stream))
    _raise(rc, "dcp_decode_partial_all_mtp")


def dcp_attention_all(desc: AttnDesc, q: torch.Tensor, shards, seq_lens: torch.Tensor, shard_starts: torch.Tensor,
                      o_parts: torch.Tensor, lses: torch.Tensor, o: torch.Tensor, lse_out: torch.Tensor | None,
                      workspace: torch.Tensor, err: torch.Tensor | None = None, stream=None):
    """Partial attention of every shard and the merge in one call. q is
    [B, Hq, Dk] (one-token decode) or [B, q_len, Hq, Dk]; o_parts / lses are
    scratch of the shards' partial rows; o [B, (q_len,) Hq, Dv], lse_out
    [B, (q_len,) Hq] or None receive the merged result."""
    _check(q, torch.bfloat16, "q")
    _check(seq_lens, torch.int32, "seq_lens")
    _check(shard_starts, torch.int32, "shard_starts")
    _check(o_parts, torch.float32, "o_parts")
    _check(lses, torch.float32, "lses")
    _check(o, torch.float32, "o")
    if lse_out is not None:
        _check(lse_out, torch.float32, "lse_out")
    _check(workspace, torch.uint8, "workspace")
    if err is not None:
        _check(err, torch.int32, "err")
    q_len = 1 if q.dim() == 3 else int(q.shape[1])
    arr = _shards(shards)
    rc = load().dcp_attention_all(ctypes.byref(desc._c), q.data_ptr(), arr, len(shards), seq_lens.data_ptr(),
                                  shard_starts.data_ptr(), int(q.shape[0]), q_len, o_parts.data_ptr(),
                                  lses.data_ptr(), o.data_ptr(), _ptr(lse_out), workspace.data_ptr(),
                                  workspace.numel(), _ptr(err), _stream(stream))
    _raise(rc, "dcp_attention_all")


def dcp_decode_partial_all_noalloc(desc: AttnDesc, q: torch.Tensor, shards, seq_lens: torch.Tensor,
                                   shard_starts: torch.Tensor, o_parts: torch.Tensor, lses: torch.Tensor,
                                   err: torch.Tensor | None = None, stream=None):
    """dcp_decode_partial_all without a caller workspace: the library's fixed
    device scratch (DCP_NOALLOC_SCRATCH_BYTES) is used instead."""
    _check(q, torch.bfloat16, "q")
    _check(seq_lens, torch.int32, "seq_lens")
    _check(shard_starts, torch.int32, "shard_starts")
    _check(o_parts, torch.float32, "o_parts")
    _check(lses, torch.float32, "lses")
    if err is not None:
        _check(err, torch.int32, "err")
    arr = _shards(shards)
    rc = load().dcp_decode_partial_all_noalloc(ctypes.byref(desc._c), q.data_ptr(), arr, len(shards),
                                               seq_lens.data_ptr(), shard_starts.data_ptr(), int(q.shape[0]),
                                               o_parts.data_ptr(), lses.data_ptr(), _ptr(err), _stream(stream))
    _raise(rc, "dcp_decode_partial_all_noalloc")


def dcp_merge(o_parts: torch.Tensor, lses: torch.Tensor, o: torch.Tensor, lse_out: torch.Tensor | None = None,
              stream=None):
    """o_parts [N, ..., Hq, Dv] fp32, lses [N, ..., Hq] fp32 -> o [..., Hq, Dv] (+ lse_out [..., Hq]);
    the middle dimensions (sequences, or sequences x query tokens) are merged row by row."""
    _check(o_parts, torch.float32, "o_parts")
    _check(lses, torch.float32, "lses")
    _check(o, torch.float32, "o")
    if lse_out is not None:
        _check(lse_out, torch.float32, "lse_out")
    if o_parts.dim() < 4:
        raise ValueError("o_parts must be [N, ..., Hq, Dv]")
    N, Hq, Dv = int(o_parts.shape[0]), int(o_parts.shape[-2]), int(o_parts.shape[-1])
    B = o_parts.numel() // max(1, N * Hq * Dv)
    rc = load().dcp_merge(o_parts.data_ptr(), lses.data_ptr(), N, B, Hq, Dv, o.data_ptr(), _ptr(lse_out),
                          _stream(stream))
    _raise(rc, "dcp_merge")


# ---------------------------------------------------------------------------
# cache rows, attention weight and eviction
# ---------------------------------------------------------------------------
def _check_shape(t: torch.Tensor, dtype, shape, name: str, device):
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == device and t.shape == shape and t.is_contiguous():
        return
    _check(t, dtype, name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")


def _cache(desc: AttnDesc, shards, device, batch: int) -> ctypes.Array:
    """The shards for the library, whose pools and tables have the descriptor's
    types and shapes and one device, the current one."""
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a CUDA device, not on {device}")
    if device.index != _current_device():
        raise ValueError(f"tensors are on {device}, the current device is cuda:{_current_device()}")
    want = (device, desc.kv_torch_dtype, batch, *desc.block_shapes)
    forms = [s._form() for s in shards]
    for i, form in enumerate(forms):
        if form[2] != want:
            for name, got, need in zip(("device", "pool type", "block_table rows", "k_pool block", "v_pool block"), form[2], want):
                if got != need:
                    raise ValueError(f"shards[{i}]: {name} must be {need}, got {got}")
    return _array(shards, forms)


def _check_err(err, device):
    if err is not None:
        _check(err, torch.int32, "err")
        if err.numel() < 1 or err.device != device:
            raise ValueError("err must hold one int32 on the tensors' device")


def dcp_kv_read(desc: AttnDesc, shards, shard_starts: torch.Tensor, positions: torch.Tensor, k_out: torch.Tensor,
                v_out: torch.Tensor | None = None, seq_ids: torch.Tensor | None = None,
                err: torch.Tensor | None = None, stream=None):
    """Cached rows of tokens (seq_ids[j], positions[j]) as bf16: k_out and
    v_out [T, Hkv, D] (MLA: k_out [T, Dk], v_out None)."""
    _check(shard_starts, torch.int32, "shard_starts")
    _check(positions, torch.int32, "positions")
    B, T, dev = int(shard_starts.shape[0]), int(positions.numel()), positions.device
    arr = _cache(desc, shards, dev, B)
    _check_shape(shard_starts, torch.int32, (B, len(shards)), "shard_starts", dev)
    if seq_ids is not None:
        _check_shape(seq_ids, torch.int32, (T,), "seq_ids", dev)
    mla = desc.kind == DCP_KIND_MLA
    _check_shape(k_out, torch.bfloat16, (T, desc.head_dim_k) if mla else (T, desc.num_kv_heads, desc.head_dim_k),
                 "k_out", dev)
    if v_out is not None:
        _check_shape(v_out, torch.bfloat16, (T, desc.num_kv_heads, desc.head_dim_v), "v_out", dev)
    _check_err(err, dev)
    rc = load().dcp_kv_read(ctypes.byref(desc._c), arr, len(shards), shard_starts.data_ptr(), B,
                            _ptr(seq_ids), positions.data_ptr(), k_out.data_ptr(), _ptr(v_out), T, _ptr(err),
                            _stream(stream))
    _raise(rc, "dcp_kv_read")


def dcp_attention_mass(desc: AttnDesc, q: torch.Tensor, shards, seq_lens: torch.Tensor, shard_starts: torch.Tensor,
                       lse: torch.Tensor, mass_out: torch.Tensor, mass_in: torch.Tensor | None = None,
                       err: torch.Tensor | None = None, stream=None):
    """Attention weight of every cached token: mass_out[b, h, t] = mass_in[b, h,
    t] (tokens cached before the step) + sum of exp(scale q.k_t - lse) over the
    step's query tokens and KV head h's query heads. q [B, (q_len,) Hq, Dk],
    lse [B, (q_len,) Hq] of the step's attention, masses [B, Hkv, max_tokens]
    fp32; mass_in None counts as zero and may be mass_out."""
    _check(q, torch.bfloat16, "q")
    if q.dim() not in (3, 4):
        raise ValueError("q must be [B, Hq, Dk] or [B, q_len, Hq, Dk]")
    B, dev = int(q.shape[0]), q.device
    q_len = 1 if q.dim() == 3 else int(q.shape[1])
    rows = (B,) if q.dim() == 3 else (B, q_len)
    arr = _cache(desc, shards, dev, B)
    _check_shape(q, torch.bfloat16, (*rows, desc.num_q_heads, desc.head_dim_k), "q", dev)
    _check_shape(lse, torch.float32, (*rows, desc.num_q_heads), "lse", dev)
    _check_shape(seq_lens, torch.int32, (B,), "seq_lens", dev)
    _check_shape(shard_starts, torch.int32, (B, len(shards)), "shard_starts", dev)
    cap = int(mass_out.shape[-1]) if mass_out.dim() else 0
    _check_shape(mass_out, torch.float32, (B, desc.num_kv_heads, cap), "mass_out", dev)
    if mass_in is not None:
        _check_shape(mass_in, torch.float32, (B, desc.num_kv_heads, cap), "mass_in", dev)
    _check_err(err, dev)
    rc = load().dcp_attention_mass(ctypes.byref(desc._c), q.data_ptr(), arr, len(shards),
                                   seq_lens.data_ptr(), shard_starts.data_ptr(), B, q_len, lse.data_ptr(),
                                   _ptr(mass_in), mass_out.data_ptr(), cap, _ptr(err), _stream(stream))
    _raise(rc, "dcp_attention_mass")


def dcp_evict_workspace_size(desc: AttnDesc, batch: int, n_shards: int, max_tokens: int) -> int:
    return int(load().dcp_evict_workspace_size(ctypes.byref(desc._c), batch, n_shards, max_tokens))


def dcp_kv_evict(desc: AttnDesc, shards, seq_lens: torch.Tensor, shard_starts: torch.Tensor, keep: torch.Tensor,
                 n_sink: int, n_recent: int, mass_in: torch.Tensor, mass_out: torch.Tensor, pos_out: torch.Tensor,
                 new_starts: torch.Tensor, new_lens: torch.Tensor, workspace: torch.Tensor,
                 pos_in: torch.Tensor | None = None, known_lens: torch.Tensor | None = None,
                 total_lens: torch.Tensor | None = None, err: torch.Tensor | None = None, stream=None):
    """Keep the keep[b, i] heaviest tokens of every (sequence, shard, KV head),
    moving their rows to the front of the shard in place. mass_in, mass_out
    [B, Hkv, max_tokens] fp32, pos_in, pos_out the same int32, keep and
    new_starts [B, N], the lengths [B] int32; outputs are other tensors than
    inputs. Go on with new_starts and new_lens."""
    _check(shard_starts, torch.int32, "shard_starts")
    B, N, dev = int(shard_starts.shape[0]), len(shards), shard_starts.device
    arr = _cache(desc, shards, dev, B)
    cap = int(mass_in.shape[-1]) if mass_in.dim() else 0
    for name, count in (("n_sink", n_sink), ("n_recent", n_recent)):
        if not -1 << 31 <= count < 1 << 31:
            raise ValueError(f"{name} must fit 32 bits, got {count}")
    i32, rows = torch.int32, (B, desc.num_kv_heads, cap)
    _check_shape(shard_starts, i32, (B, N), "shard_starts", dev)
    _check_shape(seq_lens, i32, (B,), "seq_lens", dev)
    _check_shape(keep, i32, (B, N), "keep", dev)
    _check_shape(mass_in, torch.float32, rows, "mass_in", dev)
    _check_shape(mass_out, torch.float32, rows, "mass_out", dev)
    _check_shape(pos_out, i32, rows, "pos_out", dev)
    _check_shape(new_starts, i32, (B, N), "new_starts", dev)
    _check_shape(new_lens, i32, (B,), "new_lens", dev)
    if pos_in is not None:
        _check_shape(pos_in, i32, rows, "pos_in", dev)
    if known_lens is not None:
        _check_shape(known_lens, i32, (B,), "known_lens", dev)
    if total_lens is not None:
        _check_shape(total_lens, i32, (B,), "total_lens", dev)
    _check(workspace, torch.uint8, "workspace")
    if workspace.device != dev:
        raise ValueError(f"workspace is on {workspace.device}, not on {dev}")
    _check_err(err, dev)
    rc = load().dcp_kv_evict(ctypes.byref(desc._c), arr, N, seq_lens.data_ptr(), shard_starts.data_ptr(),
                             B, keep.data_ptr(), n_sink, n_recent, mass_in.data_ptr(), _ptr(pos_in),
                             _ptr(known_lens), _ptr(total_lens), cap, mass_out.data_ptr(), pos_out.data_ptr(),
                             new_starts.data_ptr(), new_lens.data_ptr(), workspace.data_ptr(), workspace.numel(),
                             _ptr(err), _stream(stream))
    _raise(rc, "dcp_kv_evict")
