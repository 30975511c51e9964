"""Attention rows whose weight is spread over many binades: a token that takes
nearly all of it and holds next to nothing, and many light tokens whose values
are then the output. Every output is bounded by the weights and values of its
own dim, not by the cache's largest value."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from compress_helpers import Cache, as_cached, queries
from helpers import f64

pytestmark = pytest.mark.gpu

GRID = np.array([1.0, 1.5, 2.0, 3.0])  # exact in every cache type under a block maximum of 3


def _bf16(x):
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).to(torch.bfloat16)


def _rows(kv, n, hkv, d, key, values):
    """bf16 rows whose score is key [n, hkv] times the query's one entry, and values [n, hkv, dv]."""
    if d == 576:  # one row: the value and, behind it, the key's dims
        row = np.zeros((n, 1, d))
        row[..., :512] = values
        row[..., 512] = key
        return _bf16(row), None
    k = np.zeros((n, hkv, d))
    k[..., 0] = key
    return _bf16(k), _bf16(values)


def _query(J, hq, d, a):
    q = torch.zeros(1, J, hq, d, dtype=torch.bfloat16)
    q[..., 512 if d == 576 else 0] = torch.as_tensor(a, dtype=torch.float32).to(torch.bfloat16)
    return q


def _reference(q, K, V, n):
    """(o, lse, sum_t p_t |v_t|) of the query tokens in float64; scale 1."""
    o, lse = O.mtp_attention(q, K, V, 1.0, n)
    mag, _ = O.mtp_attention(q, K, np.abs(V), 1.0, n)
    return o, lse, mag


# Relative error of a light token's weight in O. bf16: P as two bf16 terms
# (2^-16 with the truncated second). 4 bits: two fp16 terms, of which a token
# 2^-25 of its neighbours' largest keeps 2^-14, or two bf16 terms where scales
# are far apart. 8 bits: one fp16 term (2^-12) down to 2^-14 of its range, 2^-11
# at half that.
REL = {"bf16": 2.0 ** -15, "mxfp4": 2.0 ** -13, "fp8": 2.0 ** -10}


def _bound(kv, mag, n, binades, d=0):
    """Beside P: the log2 argument's rounding (binades 2^-23 ln 2, numerator and denominator) and exp2's 2^-22 each, and
    the fp32 sums over the tokens."""
    return mag * (REL[kv] + 2 * (binades * 2.0 ** -23 + 2.0 ** -22) + (n + 8) * 2.0 ** -23)


@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("kv,hq,hkv,d,bs,n,J", [
    ("bf16", 8, 2, 64, 16, 180, 1),
    ("bf16", 16, 1, 128, 16, 4000, 1),
    ("bf16", 128, 1, 576, 64, 4000, 1),
    ("mxfp4", 2, 1, 64, 16, 180, 1),      # one CTA's run, rows of a lane half empty
    ("mxfp4", 16, 1, 64, 16, 180, 1),
    ("mxfp4", 8, 2, 128, 16, 180, 1),
    ("mxfp4", 64, 2, 128, 32, 170, 1),
    ("mxfp4", 8, 1, 128, 16, 180, 3),
    ("mxfp4", 16, 1, 128, 16, 20000, 1),
    ("fp8", 8, 2, 64, 16, 180, 1),
    ("fp8", 16, 1, 128, 16, 4000, 1),
    ("fp8", 8, 1, 128, 16, 180, 4),
    ("fp8", 128, 1, 576, 64, 180, 1),
    ("fp8", 128, 1, 576, 64, 4000, 2),
])
def test_light_tokens_behind_an_empty_sink(kv, hq, hkv, d, bs, n, J, where):
    """A token 17.375 nats above all others holds a zero value: the output is the light tokens' share, 2^-25 each."""
    dv = 512 if d == 576 else d
    at = {"first": 0, "middle": n // 2, "last": n - J}[where]   # every query token sees it
    key = np.zeros((n, hkv))
    key[at] = 4.0
    values = np.broadcast_to(GRID[np.arange(dv) % 4], (n, hkv, dv)).copy()
    values[at] = 0.0
    k, v = _rows(kv, n, hkv, d, key, values)
    c = Cache(kv, [n], hq, hkv, d, bs, 1, [(k, v)], scale=1.0)
    q = _query(J, hq, d, 17.375 / 4)
    o, lse = c.attend(q.cuda())
    assert c.flag() == 0
    K = as_cached(kv, k)
    V = K[..., :512] if d == 576 else as_cached(kv, v)
    assert np.array_equal(V, values) and np.array_equal(K[..., 512 if d == 576 else 0], key)
    ro, rl, mag = _reference(f64(q[0]), K, V, n)
    err = np.abs(o[0].cpu().numpy() - ro)
    tol = _bound(kv, mag, n, 26)
    assert (err <= tol).all(), (err / mag).max()
    assert np.abs(lse[0].cpu().numpy() - rl).max() <= 1e-4


@pytest.mark.parametrize("hq,hkv,d,bs,n,J", [(2, 1, 64, 16, 700, 1), (16, 1, 128, 16, 900, 1), (32, 2, 128, 32, 333, 1),
                                             (4, 1, 64, 48, 400, 4), (16, 1, 128, 16, 30000, 1), (8, 1, 128, 64, 5000, 2)])
def test_weights_over_many_binades(hq, hkv, d, bs, n, J):
    """Scores 0 to -60 nats apart, each head at its own size, in any order: rounds of tokens that are light for one row
    and heavy for another, and maxima that rise by tens of binades late."""
    g = np.random.default_rng(n + hq)
    steps = np.array([0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
    key = -g.choice(steps, (n, hkv)) * np.exp2(g.integers(-2, 2, (n, hkv)))
    key[g.random((n, hkv)) < 0.5] = -12.0                       # most of them light
    key[: n // 2] = np.minimum(key[: n // 2], -6.0)              # the heavy ones in the second half
    values = g.choice(GRID, (n, hkv, d)) * np.exp2(g.integers(-3, 4, (n, hkv, 1)))
    k, v = _rows("mxfp4", n, hkv, d, key, values)
    c = Cache("mxfp4", [n], hq, hkv, d, bs, 1, [(k, v)], scale=1.0)
    a = 0.25 * (1 + np.arange(hq) % 8)
    q = _query(J, hq, d, np.broadcast_to(a, (J, hq)).copy())
    o, lse = c.attend(q.cuda())
    assert c.flag() == 0
    K, V = as_cached("mxfp4", k), as_cached("mxfp4", v)
    ro, rl, mag = _reference(f64(q[0]), K, V, n)
    # a token shares its operands' range with the heaviest of its 64 neighbours: 2^-39 of that is lost, whatever it is
    floor = np.abs(V).max() * 2.0 ** -38 * n
    assert (np.abs(o[0].cpu().numpy() - ro) <= _bound("mxfp4", mag, n, 40) + floor).all()
    assert np.abs(lse[0].cpu().numpy() - rl).max() <= 1e-3


@pytest.mark.parametrize("hq,hkv,d,bs,J", [(2, 1, 64, 16, 1), (16, 1, 64, 16, 1), (8, 2, 128, 16, 1), (16, 1, 128, 32, 1),
                                           (8, 1, 128, 16, 4)])
@pytest.mark.parametrize("n", [16, 33, 64, 200, 700])
def test_heavy_tokens_with_far_smaller_values(hq, hkv, d, bs, J, n):
    """One or two tokens hold nearly all of the weight, at varying places of a tile; their value blocks of 32 dims are
    up to 2^-22 of the light tokens', each block by its own factor, so that a round holds near and far scales and the
    output is the far ones'."""
    g = np.random.default_rng(1000 * d + 10 * n + hq + J)
    heavy = g.choice(n - J + 1, size=1 + n % 2, replace=False)
    key = np.zeros((n, hkv))
    key[heavy] = 4.0
    values = g.choice(GRID, (n, hkv, d)) * np.where(g.random((n, hkv, d)) < 0.5, -1.0, 1.0)
    down = np.exp2(-g.integers(0, 23, (1, hkv, d // 32, 1)).astype(float))
    at = values[heavy].reshape(len(heavy), hkv, d // 32, 32)
    values[heavy] = (np.abs(at) * down).reshape(len(heavy), hkv, d)
    k, v = _rows("mxfp4", n, hkv, d, key, values)
    c = Cache("mxfp4", [n], hq, hkv, d, bs, 1, [(k, v)], scale=1.0)
    q = _query(J, hq, d, 5.25)                                  # 21 nats: 30 binades
    o, lse = c.attend(q.cuda())
    assert c.flag() == 0
    K, V = as_cached("mxfp4", k), as_cached("mxfp4", v)
    ro, rl, mag = _reference(f64(q[0]), K, V, n)
    # heavy tokens keep two bf16 terms at least; light ones, 2^-30, the operands' floor of 2^-39
    tol = _bound("bf16", mag, n, 31) + 3.0 * n * 2.0 ** -38
    err = np.abs(o[0].cpu().numpy() - ro)
    assert (err <= tol).all(), (err / mag).max()
    assert np.abs(lse[0].cpu().numpy() - rl).max() <= 1e-4


def test_uniform_queries_are_unchanged_by_a_common_offset():
    """Scores of any common size give the same weights: all equal, the mean of the values."""
    n, hq, d = 500, 8, 64
    values = np.broadcast_to(GRID[np.arange(d) % 4], (n, 1, d)) * np.where(np.arange(n) % 2, 1.0, 0.5)[:, None, None]
    for size in (-6.0, 0.0, 6.0):
        k, v = _rows("mxfp4", n, 1, d, np.full((n, 1), size), values)
        c = Cache("mxfp4", [n], hq, 1, d, 16, 1, [(k, v)], scale=1.0)
        o, lse = c.attend(_query(1, hq, d, 16.0).cuda())
        assert np.abs(o[0].cpu().numpy() - values.mean(axis=0)).max() <= 3.0 * (2.0 ** -15 + (n + 8) * 2.0 ** -23)
        assert np.abs(lse[0].cpu().numpy() - (16.0 * size + math.log(n))).max() <= 1e-3 and c.flag() == 0


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("size", [1.1e3, 3.7e5, 1.3e7, 9.1e8])
@pytest.mark.parametrize("kv,hq,hkv,d,bs,J", [("mxfp4", 8, 2, 64, 16, 1), ("mxfp4", 16, 1, 128, 16, 1), ("mxfp4", 4, 1, 128, 16, 5),
                                              ("fp8", 8, 2, 64, 16, 1), ("fp8", 128, 1, 576, 64, 1), ("bf16", 16, 1, 128, 16, 1),
                                              ("bf16", 128, 1, 576, 64, 1)])
def test_scores_past_the_fractions_of_fp32(kv, hq, hkv, d, bs, J, size, sign):
    """Scores whose spacing in fp32 is many binades: the largest ones share the weight, the others have none, and nothing
    overflows on the way. The largest ones' tokens hold the same values: a sequence is cut into pieces whose weights
    come from their fp32 LSEs, spaced 2^-5 (size 3.7e5) to 64 nats (9.1e8) here, so that the pieces' shares of the
    weight are not determined, only their sum."""
    n, dv = 500, 512 if d == 576 else d
    g = np.random.default_rng(int(size))
    key = sign * g.choice([0.5, 1.0, 1.5, 2.0, 3.0], (n, hkv))
    top = [7, 300, 301, 470]                                     # in rounds, warps and shards of their own
    key[top] = sign * 4.0
    values = g.choice(GRID, (n, hkv, dv))
    values[top] = values[7]
    k, v = _rows(kv, n, hkv, d, key, values)
    c = Cache(kv, [n], hq, hkv, d, bs, 2, [(k, v)], scale=sign * size / 3.0)
    o, lse = c.attend(_query(J, hq, d, 0.75).cuda())
    assert c.flag() == 0
    want = np.repeat(values[7], hq // hkv, axis=0)
    got = o[0].cpu().numpy()
    assert np.abs(got - want).max() <= 3.0 * (REL[kv] + (n + 8) * 2.0 ** -23), np.abs(got - want).max()
    assert np.abs(lse[0].cpu().numpy() - size).max() <= math.log(len(top)) + 2.0 ** -20 * size


@pytest.mark.parametrize("kv,hq,hkv,d,bs", [("mxfp4", 8, 1, 64, 16), ("mxfp4", 16, 1, 128, 16), ("fp8", 8, 1, 64, 16),
                                            ("fp8", 16, 1, 128, 16), ("fp8", 128, 1, 576, 64)])
def test_large_scores_a_step_of_fp32_apart(kv, hq, hkv, d, bs):
    """Scores near 2^30 that rise by single steps of fp32 (64 nats and more in all) from token to token, whose rounded
    products with the scale may be equal: the outputs stay finite and within the values."""
    n, dv = 400, 512 if d == 576 else d
    g = np.random.default_rng(d)
    at = 512 if d == 576 else 0
    k = np.zeros((n, hkv, d))
    k[..., at] = 4.0
    k[..., at + 1] = np.linspace(-1, 1, n)[:, None]       # a few steps of fp32 beside the first product
    values = g.choice(GRID, (n, hkv, dv))
    if d == 576:
        k[..., :512] = values
    c = Cache(kv, [n], hq, hkv, d, bs, 1, [(_bf16(k), None if d == 576 else _bf16(values))], scale=1.43e9 / 4)
    q = torch.zeros(1, 1, hq, d, dtype=torch.bfloat16)
    q[..., at] = 1.0
    q[..., at + 1] = torch.exp2(-torch.arange(hq) / 8 - 14).to(torch.bfloat16)
    for sign in (1.0, -1.0):
        o, lse = c.attend((q * sign).cuda())
        got = o[0].cpu().numpy()
        assert c.flag() == 0 and np.isfinite(got).all()
        assert got.min() >= 1.0 - 2.0 ** -9 and got.max() <= 3.0 + 2.0 ** -7
        assert np.abs(lse[0].cpu().numpy() - sign * 1.43e9).max() <= 2.0 ** 18


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("hq,hkv,d,J", [(8, 2, 64, 1), (16, 1, 128, 1), (4, 1, 128, 4), (40, 1, 64, 2)])
def test_a_bad_query_row_stays_by_itself(hq, hkv, d, J, bad):
    """A row of NaN or infinities gives NaN, and the rows that share its lane what they give without it."""
    lens = [300, 70]
    g = torch.Generator().manual_seed(3)
    rows = [tuple(torch.randn(n, hkv, d, generator=g).to(torch.bfloat16) for _ in range(2)) for n in lens]
    c = Cache("mxfp4", lens, hq, hkv, d, 16, 2, rows)
    q = queries(2, J, hq, d, 5)
    o, lse = c.attend(q.cuda())
    out = torch.zeros(2, J, hq, dtype=torch.bool)
    out[0, 0, 1], out[1, J - 1, hq - 1] = True, True
    q[out] = bad
    o2, lse2 = c.attend(q.cuda())
    out = out.cuda()
    assert c.flag() == 0
    assert torch.equal(o[~out], o2[~out]) and torch.equal(lse[~out], lse2[~out])
    assert torch.isnan(o2[out]).all() and torch.isnan(lse2[out]).all()
