"""How many slots a block of a 4-bit cache has, and rows of how many elements (CPU): a plane's bytes fit several pairs of the two, and a
call that takes the wrong pair reads and writes the slots of other requests without an error."""
import pytest
import torch

from block_table_contiguous_amd import kvx as K

BF16 = torch.bfloat16


def attention(cache, dim, **kw):
    q = torch.zeros(3, 4, dim, dtype=BF16)
    K.kvx_paged_attention_fp4(q, cache, torch.zeros(1, 2, dtype=torch.int32), torch.tensor([0, 3]), torch.tensor([3]), torch.zeros_like(q), **kw)


def rope(cache, dim, **kw):
    q, k = torch.zeros(3, 4, dim, dtype=BF16), torch.zeros(3, 2, dim, dtype=BF16)
    K.kvx_rope_and_cache_fp4(q, k, k.clone(), torch.zeros(1, 3, dtype=torch.int64), torch.zeros(8), [0] * 8, torch.zeros(3, dtype=torch.int64),
                             cache, torch.zeros_like(q), **kw)


def workspace(cache, dim, **kw):
    K.new_attention_workspace_fp4(torch.zeros(3, 4, dim, dtype=BF16), cache, 1, 3, 5000, **kw)


def struct(cache, dim, **kw):
    return K.fp4_cache(cache, dim, BF16, **kw)


CALLS = [attention, rope, workspace, struct]


@pytest.mark.parametrize("layout", list(K._FP4_AXES))
@pytest.mark.parametrize("call", CALLS)
def test_rows_of_another_length_than_the_cache_was_made_for(call, layout):
    cache = K.new_fp4_cache(4, 16, 2, 128, "cpu", layout)
    for dim in (32, 64, 256):
        with pytest.raises(ValueError, match="made for rows of 128 elements"):
            call(cache, dim, layout=layout)


@pytest.mark.parametrize("call", CALLS)
def test_a_block_size_that_the_planes_do_not_have(call):
    """Stated, it counts, for tensors that do not say what they were made for too (a view, a copy, a buffer of the caller's)."""
    cache = K.new_fp4_cache(4, 16, 2, 128, "cpu")
    for kv in (cache, cache[1:], cache.clone(), torch.zeros(4, 2, 2, 16 * 68, dtype=torch.uint8)):
        for dim, block in ((128, 8), (128, 32), (64, 16), (256, 16), (32, 16), (128, 0), (128, -16)):
            with pytest.raises(ValueError, match="fp4_plane_bytes"):
                call(kv, dim, block_size=block)


@pytest.mark.parametrize("call", CALLS)
def test_a_struct_of_another_block_size(call):
    c = K.fp4_cache(K.new_fp4_cache(4, 16, 2, 128, "cpu"), 128, BF16, block_size=16)
    if call is struct:
        assert (c.block_size, c.head_dim) == (16, 128)
        return
    with pytest.raises(ValueError, match="block_size"):
        call(c, 128, block_size=8)
    if call is not workspace:
        with pytest.raises(ValueError, match="must be"):
            call(c, 64)


@pytest.mark.parametrize("block,dim", [(1, 32), (16, 128), (24, 96), (3, 256), (100, 64), (7, 160)])
def test_the_right_sizes_are_taken(block, dim):
    cache = K.new_fp4_cache(4, block, 2, dim, "cpu")
    for kv in (cache, cache[:2], cache.clone()):
        for kw in ({}, dict(block_size=block)):
            c = K.fp4_cache(kv, dim, BF16, **kw)
            assert (c.block_size, c.head_dim, c.num_kv_heads) == (block, dim, 2)
            workspace(kv, dim, **kw)
            for call in (attention, rope):
                with pytest.raises(ValueError, match="must live on the GPU"):  # the last check of all
                    call(kv, dim, **kw)


def test_a_transfer_takes_the_16_bit_caches_sizes():
    layer, runs = torch.zeros(9, 16, 2, 2, 64, dtype=BF16), torch.zeros(4, 4, dtype=torch.int64)
    bases, count = torch.zeros(2, dtype=torch.int64), torch.zeros(1, dtype=torch.int64)
    for block, dim, says in ((16, 64, "must live on the GPU"), (8, 128, "must live on the GPU"), (8, 64, "fp4_plane_bytes"), (16, 128, "fp4_plane_bytes")):
        buf = K.new_fp4_cache(8, block, 2, dim, "cpu")  # of 8 slots of 128 elements: as many bytes, and only bytes are sent
        for call, a in ((K.kvx_pack_fp4, (bases, layer, runs, count, 4, buf)), (K.kvx_unpack_fp4, (buf, bases, layer, runs, count, 4))):
            with pytest.raises(ValueError, match=says):
                call(*a)
