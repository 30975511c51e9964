"""Read-back of an 8-bit cache rounds k_scale * decode(code) once, to bf16."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle as O
from compress_helpers import descriptor
from sequence_sharded_decode_gb300 import dcp

pytestmark = pytest.mark.gpu


def _round_to_bf16(x):
    """Nearest value of eight significant bits, ties to even (normal range), of exact float64 products."""
    m, e = np.frexp(x)
    return np.rint(m * 256.0) * np.exp2(e.astype(np.float64) - 8.0)


def _tie_scales():
    """fp32 scales whose product with some code lies just beside the middle of two bf16 values, nearer to it than fp32
    resolves."""
    found = []
    for odd in range(257, 512, 2):                     # middles between neighbouring bf16 values of [1, 2)
        middle = Fraction(odd, 256)
        for code in (1.125, 1.25, 1.375, 1.625, 1.75, 1.875):
            near = np.float32(float(middle / Fraction(code)))
            for s in (np.nextafter(near, np.float32(0)), near, np.nextafter(near, np.float32(9))):
                exact = Fraction(float(s)) * Fraction(code)
                if exact != middle and np.float32(float(s) * code) == np.float32(float(middle)):
                    found.append(float(s))
    return found[:: max(1, len(found) // 12)][:12]


@pytest.mark.parametrize("d,hkv,bs", [(64, 1, 16), (128, 2, 16), (576, 1, 64)])
@pytest.mark.parametrize("batch", [1, 32])            # many tokens per sequence; few
def test_products_beside_a_tie_round_once(d, hkv, bs, batch):
    codes = np.arange(256, dtype=np.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x38               # (NaN)
    T = 32 if batch == 32 else 40
    scales = _tie_scales()
    assert len(scales) >= 8
    wrong = 0
    for i, s in enumerate(scales):
        desc = descriptor("fp8", 128 if d == 576 else hkv, hkv, d, bs, k_scale=s, v_scale=scales[i - 1])
        ids = torch.arange(T, dtype=torch.int32) % batch
        pos = torch.arange(T, dtype=torch.int32) // batch
        rows = np.resize(np.roll(codes, 7 * i), (2, T, hkv, d))
        pools = [torch.zeros(x, dtype=torch.uint8, device="cuda") if x else None for x in desc.pool_shapes(batch * 4)]
        table = torch.arange(batch * 4, dtype=torch.int32, device="cuda").view(batch, 4)
        shards = [dcp.Shard(pools[0], pools[1], table)]
        starts, err = torch.zeros(batch, 1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        shape = (T, d) if d == 576 else (T, hkv, d)
        dev = [torch.from_numpy(rows[j]).reshape(shape).cuda() for j in range(2)]
        ids, pos = ids.cuda(), pos.cuda()
        dcp.dcp_kv_append(desc, shards, starts, pos, dev[0], None if d == 576 else dev[1], seq_ids=ids, err=err)
        out = [torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        dcp.dcp_kv_read(desc, shards, starts, pos, out[0], None if d == 576 else out[1], seq_ids=ids, err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        for j, scale in enumerate((desc.k_scale, desc.v_scale)[: 1 if d == 576 else 2]):
            exact = float(np.float32(scale)) * O.e4m3_to_f64(rows[j])      # 28 bits: exact
            want = _round_to_bf16(exact)
            wrong += int((out[j].cpu().double().numpy().reshape(want.shape) != want).sum())
    assert wrong == 0


@pytest.mark.parametrize("scale", [2.0 ** -140, 1.7 * 2.0 ** -128, 2.0 ** -126, 3e38, 1e36])
def test_scales_at_the_ends_of_the_range(scale):
    """Subnormal products, and products that overflow bf16, round like any other."""
    desc = descriptor("fp8", 1, 1, 64, 16, k_scale=scale, v_scale=scale)
    codes = torch.arange(128, dtype=torch.uint8).clamp(max=126).view(2, 1, 64).cuda()
    pools = [torch.zeros(x, dtype=torch.uint8, device="cuda") for x in desc.pool_shapes(1)]
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    shards, starts = [dcp.Shard(pools[0], pools[1], i32(0).view(1, 1))], i32(0).view(1, 1)
    dcp.dcp_kv_append(desc, shards, starts, i32(0, 1), codes, codes, seq_ids=i32(0, 0))
    out = [torch.empty(2, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    dcp.dcp_kv_read(desc, shards, starts, i32(0, 1), out[0], out[1], seq_ids=i32(0, 0))
    exact = float(np.float32(scale)) * O.e4m3_to_f64(codes.cpu().numpy())
    m, e = np.frexp(exact)
    q = np.exp2(np.maximum(e - 8, -133).astype(np.float64))               # spacing of bf16: 2^-133 for subnormals
    want = np.rint(exact / q) * q
    want = np.where(want > float(torch.finfo(torch.bfloat16).max), np.inf, want)
    for got in out:
        assert np.array_equal(got.cpu().double().numpy(), want)
