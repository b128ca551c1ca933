"""The calls of include/kvx_fp4.h without a GPU: exported, and every bad argument refused on the host before
anything is enqueued."""
import ctypes
import os
import re

import pytest
import torch

from block_table_contiguous_amd import kvx as K

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "kvx_fp4.h")
P = 0x10000  # a fake, aligned, non-null device address: never dereferenced here
OK, INVALID, MISALIGNED = K.KVX_SUCCESS, K.KVX_ERR_INVALID_ARGUMENT, K.KVX_ERR_MISALIGNED


def test_declared_symbols_are_exported_and_bound():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(kvx_[a-z_0-9]+)\s*\(", text)))
    assert names == sorted(["kvx_fp4_plane_bytes", "kvx_rope_and_cache_fp4", "kvx_paged_attention_fp4",
                            "kvx_paged_attention_fp4_workspace", "kvx_pack_fp4", "kvx_unpack_fp4"])
    for n in names:
        assert hasattr(K.LIB, n) and n in K.SIGNATURES
    assert ctypes.sizeof(K.Fp4Cache) == 5 * 8 + 4 * 4


def fp4(**kw):
    a = dict(base=P, num_blocks=100, block_stride_bytes=4 * 1088, kv_stride_bytes=1088, head_stride_bytes=2 * 1088, block_size=16,
             num_kv_heads=2, head_dim=128, dtype=0)
    a.update(kw)
    return K.Fp4Cache(**a)


def wide(**kw):
    a = dict(base=None, num_blocks=100, block_stride_bytes=8192 * 2, token_stride_bytes=1024, kv_stride_bytes=512,
             head_stride_bytes=256, block_size=16, num_kv_heads=2, head_dim=128, dtype=0)
    a.update(kw)
    return K.PagedCache(**a)


def batch(**kw):
    a = dict(block_table=P, q_offsets=P, context_lens=P, max_blocks_per_req=8, bt_row_stride=8, num_tokens=0,
             max_query_len=1, max_context_len=128, num_reqs=3)
    a.update(kw)
    return K.Batch(**a)


BAD_CACHES = [dict(num_blocks=-1), dict(num_blocks=1 << 31), dict(block_size=0), dict(num_kv_heads=0), dict(num_kv_heads=65536),
              dict(head_dim=0), dict(head_dim=16), dict(head_dim=80), dict(head_dim=120), dict(head_dim=288), dict(dtype=2),
              dict(dtype=-1), dict(block_stride_bytes=-16), dict(block_stride_bytes=1 << 52), dict(kv_stride_bytes=1 << 57),
              dict(head_stride_bytes=-16)]
ODD_CACHES = [dict(block_stride_bytes=8), dict(kv_stride_bytes=4), dict(head_stride_bytes=1090)]


@pytest.mark.parametrize("block,dim,want", [(16, 128, 1088), (1, 32, 32), (24, 96, 1232), (16, 256, 2176), (0, 128, -1), (16, 80, -1),
                                            (16, 288, -1), (-3, 64, -1), ((1 << 31) - 1, 256, ((1 << 31) - 1) * 136 + 8)])
def test_plane_bytes(block, dim, want):
    assert K._F["kvx_fp4_plane_bytes"](block, dim) == want


def attend(c=None, b=None, q=P, qt=2048, qh=256, H=4, scale=0.1, window=0, out=P, ot=2048, oh=256, lse=P, ws=None, wsb=0):
    c = fp4() if c is None else c
    b = batch() if b is None else b
    return K._F["kvx_paged_attention_fp4"](ctypes.byref(c), ctypes.byref(b), q, qt, qh, H, scale, 1, window, out, ot, oh, lse, ws,
                                           wsb, None, None)


def test_attention_refusals():
    for kw in BAD_CACHES:
        assert attend(c=fp4(**kw)) == INVALID, kw
    for kw in ODD_CACHES:
        assert attend(c=fp4(**kw)) == MISALIGNED, kw
    for kw in (dict(num_reqs=-1), dict(num_reqs=65536), dict(num_tokens=-1), dict(num_tokens=1 << 29),
               dict(max_blocks_per_req=9), dict(max_blocks_per_req=1 << 28, bt_row_stride=1 << 28),
               dict(max_query_len=-1), dict(max_context_len=-1)):
        assert attend(b=batch(**kw)) == INVALID, kw
    assert attend(H=0) == INVALID and attend(H=3) == INVALID  # not a multiple of the KV heads
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert attend(scale=scale) == INVALID, scale
    assert attend(window=-1) == INVALID
    assert attend(qt=8) == MISALIGNED and attend(qh=24) == MISALIGNED and attend(qt=-16) == INVALID
    one = batch(num_tokens=4)
    assert attend(b=one, q=None) == INVALID and attend(b=one, q=P + 8) == MISALIGNED
    assert attend(b=one, c=fp4(base=None)) == INVALID and attend(b=one, c=fp4(base=P + 8)) == MISALIGNED
    for f in ("block_table", "q_offsets", "context_lens"):
        assert attend(b=batch(num_tokens=4, **{f: None})) == INVALID, f
    assert attend(b=one, out=None) == INVALID and attend(b=one, out=P + 8) == MISALIGNED
    assert attend(b=one, ot=2056) == MISALIGNED and attend(b=one, oh=-16) == INVALID
    assert attend(b=one, ws=P + 8, wsb=64) == MISALIGNED and attend(b=one, wsb=-1) == INVALID
    # empty work never reaches the device
    assert attend(b=batch(num_tokens=0), q=None) == OK
    assert attend(b=batch(num_tokens=4, num_reqs=0), q=None) == OK


def test_workspace_sizes():
    def size(c=None, H=4, **kw):
        c = fp4() if c is None else c
        return K._F["kvx_paged_attention_fp4_workspace"](ctypes.byref(c), ctypes.byref(batch(**kw)), H)
    assert size(num_tokens=0) == 0
    assert size(num_tokens=3) >= 0 and size(num_tokens=3, max_context_len=100000) > 0
    assert size(c=fp4(head_dim=80), num_tokens=3) == -1 and size(H=3, num_tokens=3) == -1
    assert size(num_tokens=-1) == -1
    one, top = fp4(num_kv_heads=1), (1 << 31) - 65537
    assert size(c=one, H=1, num_tokens=top + 1) == -1 and size(c=one, H=1, num_tokens=top - 3 * 128) >= 0


def rope(c=None, q=P, H=4, k=P, v=2 * P, T=5, pos=P, axes=2, axis=None, freq=P, rot=64, slots=P, out=P, ko=None, vo=None, qt=2048,
         kt=512, oh=256, kot=512):
    c = fp4() if c is None else c
    axis = [0, 1] * 64 if axis is None else axis
    arr = (ctypes.c_int32 * len(axis))(*axis) if axis != "null" else None
    return K._F["kvx_rope_and_cache_fp4"](ctypes.byref(c), q, qt, 256, H, k, kt, 256, v, 512, 256, T, pos, axes, arr, freq, rot, 0,
                                          slots, out, 2048, oh, ko, kot, 256, vo, 512, 256, None, None)


def test_rope_refusals():
    for kw in BAD_CACHES:
        assert rope(c=fp4(**kw)) == INVALID, kw
    for kw in ODD_CACHES:
        assert rope(c=fp4(**kw), rot=16) == MISALIGNED, kw
    for rot in (0, 8, 24, 144, -16):
        assert rope(rot=rot) == INVALID, rot
    for axes in (0, 5, -1):
        assert rope(axes=axes) == INVALID, axes
    assert rope(axis=[2] * 64) == INVALID and rope(axis=[-1] * 64) == INVALID and rope(axis="null") == INVALID
    assert rope(T=-1) == INVALID and rope(T=1 << 22) == INVALID and rope(H=-1) == INVALID
    for kw in (dict(q=None), dict(out=None), dict(k=None), dict(v=None), dict(pos=None), dict(freq=None), dict(slots=None),
               dict(ko=3 * P), dict(vo=3 * P), dict(ko=P, vo=3 * P), dict(ko=3 * P, vo=2 * P), dict(ko=3 * P, vo=3 * P),
               dict(ko=3 * P, vo=4 * P, kot=-16)):
        assert rope(**kw) == INVALID, kw
    for kw in (dict(q=P + 8), dict(k=P + 2), dict(v=P + 4), dict(out=P + 8), dict(qt=2056), dict(kt=520), dict(oh=8),
               dict(ko=3 * P + 8, vo=4 * P), dict(ko=3 * P, vo=4 * P + 2), dict(ko=3 * P, vo=4 * P, kot=520)):
        assert rope(**kw) == MISALIGNED, kw
    assert rope(T=0, q=None, k=None) == OK


def pack(c=None, f=None, bases=P, L=2, runs=P, count=P, N=50):
    c, f = wide() if c is None else c, fp4() if f is None else f
    return K._F["kvx_pack_fp4"](ctypes.byref(c), bases, L, runs, count, N, ctypes.byref(f), None, None)


def unpack(c=None, f=None, bases=P, L=2, runs=P, count=P, N=50):
    c, f = wide() if c is None else c, fp4() if f is None else f
    return K._F["kvx_unpack_fp4"](ctypes.byref(f), ctypes.byref(c), bases, L, runs, count, N, None, None)


@pytest.mark.parametrize("fn", [pack, unpack])
def test_most_blocks_of_a_launch(fn):
    """Blocks of one piece of 128 groups: 2^27 - 8 are taken (the odd base is looked at behind the sizes), one more is not."""
    c = wide(num_kv_heads=1, num_blocks=1, block_stride_bytes=8192)
    f = fp4(num_kv_heads=1, num_blocks=1 << 27, block_stride_bytes=2 * 1088, base=P + 8)
    assert fn(c=c, f=f, L=1, N=(1 << 27) - 8) == MISALIGNED
    assert fn(c=c, f=f, L=1, N=(1 << 27) - 7) == INVALID and fn(c=c, f=f, L=1, N=1 << 27) == INVALID


@pytest.mark.parametrize("fn", [pack, unpack])
def test_transfer_refusals(fn):
    for kw in BAD_CACHES:
        assert fn(f=fp4(**kw)) == INVALID, kw
    for kw in ODD_CACHES:
        assert fn(f=fp4(**kw)) == MISALIGNED, kw
    for kw in (dict(num_blocks=-1), dict(block_size=0), dict(head_dim=0), dict(dtype=3), dict(token_stride_bytes=-16)):
        assert fn(c=wide(**kw)) == INVALID, kw
    for kw in (dict(token_stride_bytes=1032), dict(block_stride_bytes=8)):
        assert fn(c=wide(**kw)) == MISALIGNED, kw
    # the two sides have the same sizes, and the 4-bit blocks are enough
    for kw in (dict(block_size=8), dict(head_dim=64), dict(num_kv_heads=1), dict(dtype=1), dict(num_blocks=99)):
        assert fn(f=fp4(**kw)) == INVALID, kw
    for kw in (dict(L=-1), dict(N=-1), dict(N=1 << 31), dict(L=3), dict(bases=None), dict(runs=None), dict(count=None),
               dict(f=fp4(base=None))):
        assert fn(**kw) == INVALID, kw
    big = dict(block_size=1 << 28, head_dim=256)
    assert fn(c=wide(token_stride_bytes=0, **big), f=fp4(**big)) == INVALID  # groups of a block
    for kw in (dict(runs=P + 8), dict(f=fp4(base=P + 8))):
        assert fn(**kw) == MISALIGNED, kw
    assert fn(L=0, bases=None) == OK and fn(N=0, runs=None) == OK


def test_binding_refuses_what_the_abi_cannot_see():
    with pytest.raises(ValueError):
        K.fp4_plane_bytes(16, 80)
    kv = K.new_fp4_cache(10, 16, 2, 64, "cpu")
    assert kv.shape == (10, 2, 2, 16 * 34) and K.new_fp4_cache(10, 16, 3, 64, "cpu", "kv_blocks_heads").shape == (2, 10, 3, 16 * 34)
    for err, a in [(ValueError, (kv, 96, torch.bfloat16)), (TypeError, (kv, 64, torch.float32)), (ValueError, (kv[0], 64, torch.float16)),
                   (ValueError, (kv.view(torch.int8), 64, torch.float16)), (ValueError, (kv[..., ::2], 64, torch.float16)),
                   (ValueError, (kv[..., :-1], 64, torch.float16)), (ValueError, (kv, 64, torch.float16, "blocks")),
                   (ValueError, (kv[:, :1], 64, torch.float16, "blocks_kv_heads")), (ValueError, (kv, 0, torch.float16))]:
        with pytest.raises(err):
            K.fp4_cache(*a)
    c = K.fp4_cache(kv, 64, torch.float16)
    assert (c.block_size, c.num_kv_heads, c.num_blocks, c.kv_stride_bytes, c.head_stride_bytes) == (16, 2, 10, 544, 1088)
    q = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(3, 3, dtype=torch.int32), torch.zeros(3, dtype=torch.int64)
    off = torch.zeros(4, dtype=torch.int64)
    out, lse = torch.zeros_like(q), torch.zeros(5, 4)
    for err, kw in [(TypeError, dict(kv_cache=c)), (ValueError, dict(kv_cache=kv[0])), (ValueError, dict(layout="blocks_kv_heads", kv_cache=kv[:, :1])),
                    (ValueError, dict(query=q[:, :3])), (ValueError, dict(query=q[..., :32])), (ValueError, dict(out=out[:4])),
                    (ValueError, dict(lse=lse[:4])), (ValueError, dict(block_table=table[:2])), (ValueError, dict(q_offsets=off[:3])),
                    (ValueError, dict(query=q[0])), (ValueError, {})]:  # the last: everything fits, but nothing is on a GPU
        a = dict(query=q, kv_cache=kv, block_table=table, q_offsets=off, context_lens=lens, out=out, lse=lse)
        a.update(kw)
        with pytest.raises(err):
            K.kvx_paged_attention_fp4(**a)
    k = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    pos, freq, slots = torch.zeros(2, 5, dtype=torch.int64), torch.zeros(32), torch.zeros(5, dtype=torch.int64)
    for kw in (dict(pair_axis=[0] * 31), dict(positions=pos[:, :4].contiguous()), dict(query_out=None), dict(key=q), dict(key_out=k),
               dict(query_out=out[:, :2]), dict(key_out=k[:4], value_out=k), dict()):
        a = dict(query=q, key=k, value=k, positions=pos, inv_freq=freq, pair_axis=[0] * 32, slot_mapping=slots, kv_cache=kv,
                 query_out=out)
        a.update(kw)
        with pytest.raises(ValueError):
            K.kvx_rope_and_cache_fp4(**a)
    for kw in (dict(kv_cache=c), dict(value=k.half()), dict(query=q.half()), dict(query_out=out.half()), dict(key_out=k.half(), value_out=k),
               dict(key=k.float(), kv_cache=K.fp4_cache(kv, 64, torch.bfloat16))):
        a = dict(query=q, key=k, value=k, positions=pos, inv_freq=freq, pair_axis=[0] * 32, slot_mapping=slots, kv_cache=kv,
                 query_out=out)
        a.update(kw)
        with pytest.raises(TypeError):
            K.kvx_rope_and_cache_fp4(**a)
    layer = torch.zeros(9, 16, 2, 2, 64, dtype=torch.bfloat16)
    runs, count = torch.zeros(4, 4, dtype=torch.int64), torch.zeros(1, dtype=torch.int64)
    bases = torch.zeros(2, dtype=torch.int64)
    for kw in (dict(send_buf=kv[:7]), dict(kv_cache=layer[..., :32]), dict(send_buf=K.fp4_cache(kv, 64, torch.float16)),
               dict(xfers=runs[:3]), dict(send_buf=K.new_fp4_cache(10, 8, 2, 64, "cpu")), dict()):
        a = dict(layer_bases=bases, kv_cache=layer, xfers=runs, xfer_count=count, total_blocks=4, send_buf=kv)
        a.update(kw)
        with pytest.raises(ValueError):
            K.kvx_pack_fp4(**a)
        with pytest.raises(ValueError):
            K.kvx_unpack_fp4(**a)
