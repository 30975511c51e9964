"""Shards and descriptors of the Python binding as ordinary objects: copied,
pickled and changed in place, before and after their first use."""
import copy
import pickle

import pytest
import torch

from compress_helpers import Cache, normal_rows, queries
from sequence_sharded_decode_gb300 import dcp

pytestmark = pytest.mark.gpu


def _cache():
    return Cache("bf16", [64, 40], 4, 2, 64, 16, 2, normal_rows([64, 40], 2, 64, 71))


@pytest.mark.parametrize("kind", ["copy", "deepcopy", "pickle"])
def test_used_shards_and_descriptors_are_copied(kind):
    c = _cache()
    q = queries(2, 1, 4, 64, 1).cuda()
    o, lse = c.attend(q)
    again = {"copy": copy.copy, "deepcopy": copy.deepcopy, "pickle": lambda x: pickle.loads(pickle.dumps(x))}[kind]
    c.desc, shards = again(c.desc), [again(s) for s in c.shards]
    if kind != "copy":                                    # tensors of their own: the old ones may go
        assert all(a.k_pool.data_ptr() != b.k_pool.data_ptr() for a, b in zip(shards, c.shards))
        for s in c.shards:
            s.k_pool.zero_(), s.block_table.fill_(-1)
    c.shards = shards
    o2, lse2 = c.attend(q)
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and c.flag() == 0


def test_a_copy_follows_its_own_fields():
    c = _cache()
    first = c.shards[0]
    first.c()
    other = copy.copy(first)
    other.block_table = first.block_table[:, :1].contiguous()
    assert other.c().max_blocks_per_seq == 1 and first.c().max_blocks_per_seq == first.block_table.shape[1] > 1


def test_library_forms_are_the_callers_own():
    """What c() returns may be changed; the shard's and the descriptor's later calls do not see it."""
    c = _cache()
    q = queries(2, 1, 4, 64, 2).cuda()
    o, _ = c.attend(q)
    form, desc = c.shards[0].c(), c.desc.c()
    form.k_pool, form.num_blocks, desc.num_q_heads, desc.scale = None, 0, 2, 0.0
    o2, _ = c.attend(q)
    assert torch.equal(o, o2) and c.desc.c().num_q_heads == 4 and c.shards[0].c().num_blocks == c.shards[0].k_pool.shape[0]


def test_tensors_changed_in_place_are_looked_at_again():
    c = _cache()
    shard = c.shards[0]
    shard.c()
    shard.block_table.resize_(2, 2)
    shard.c()
    shard.block_table.t_()                                 # the same storage and shape, not the same table
    with pytest.raises(ValueError, match="contiguous"):
        shard.c()
    shard.block_table.t_()
    shard.c()
    shard.k_pool.data = shard.k_pool.data.view(torch.float16)
    with pytest.raises(TypeError, match="bf16"):
        shard.c()
