"""The calls of include/kvx_attention.h without a GPU: exported, and every bad argument refused on
the host before anything is enqueued."""
import ctypes
import os
import re

import pytest
import torch

from block_table_contiguous_amd import kvx as K

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "kvx_attention.h")
P = 0x10000  # a fake, aligned, non-null device address: never dereferenced here
OK, INVALID, MISALIGNED = K.KVX_SUCCESS, K.KVX_ERR_INVALID_ARGUMENT, K.KVX_ERR_MISALIGNED


def test_declared_symbols_are_exported_and_bound():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(kvx_[a-z_0-9]+)\s*\(", text)))
    assert names == sorted(["kvx_rope_and_cache", "kvx_paged_attention", "kvx_paged_attention_workspace",
                            "kvx_attention_mass", "kvx_evict_select", "kvx_evict_compact"])
    for n in names:
        assert hasattr(K.LIB, n) and n in K.SIGNATURES
    # the structs' sizes as the header lays them out: 6 and 8 words, then the 32-bit fields
    assert ctypes.sizeof(K.PagedCache) == 6 * 8 + 4 * 4 and ctypes.sizeof(K.Batch) == 8 * 8 + 8


def cache(**kw):
    a = dict(base=P, num_blocks=100, block_stride_bytes=8192 * 2, token_stride_bytes=1024, kv_stride_bytes=512,
             head_stride_bytes=256, block_size=16, num_kv_heads=2, head_dim=128, dtype=0)
    a.update(kw)
    return K.PagedCache(**a)


def batch(**kw):
    a = dict(block_table=P, q_offsets=P, context_lens=P, max_blocks_per_req=8, bt_row_stride=8, num_tokens=0,
             max_query_len=1, max_context_len=128, num_reqs=3)
    a.update(kw)
    return K.Batch(**a)


BAD_CACHES = [dict(num_blocks=-1), dict(num_blocks=1 << 31), dict(block_size=0), dict(num_kv_heads=0), dict(head_dim=0),
              dict(head_dim=264), dict(dtype=2), dict(dtype=-1), dict(block_stride_bytes=-16),
              dict(block_stride_bytes=1 << 52), dict(token_stride_bytes=-16), dict(kv_stride_bytes=1 << 57),
              dict(head_stride_bytes=-16)]
ODD_CACHES = [dict(head_dim=20), dict(block_stride_bytes=8), dict(token_stride_bytes=1032), dict(kv_stride_bytes=4),
              dict(head_stride_bytes=40)]


def attend(c=None, b=None, q=P, qt=2048, qh=256, H=4, scale=0.1, window=0, out=P, ot=2048, oh=256, lse=P, ws=None, wsb=0):
    c = cache() if c is None else c
    b = batch() if b is None else b
    return K._F["kvx_paged_attention"](ctypes.byref(c), ctypes.byref(b), q, qt, qh, H, scale, 1, window, out, ot, oh, lse, ws,
                                       wsb, None, None)


def mass(c=None, b=None, q=P, qt=2048, qh=256, H=4, scale=0.1, window=0, lse=P, m=P, rs=1000, hs=500, w=500):
    c = cache() if c is None else c
    b = batch() if b is None else b
    return K._F["kvx_attention_mass"](ctypes.byref(c), ctypes.byref(b), q, qt, qh, H, scale, 1, window, lse, m, rs, hs, w, None,
                                      None)


@pytest.mark.parametrize("fn", [attend, mass])
def test_attention_refusals(fn):
    for kw in BAD_CACHES:
        assert fn(c=cache(**kw)) == INVALID, kw
    for kw in ODD_CACHES:
        assert fn(c=cache(**kw)) == MISALIGNED, kw
    for kw in (dict(num_reqs=-1), dict(num_reqs=65536), dict(num_tokens=-1), dict(num_tokens=1 << 29),
               dict(max_blocks_per_req=9), dict(max_blocks_per_req=1 << 28, bt_row_stride=1 << 28),
               dict(max_query_len=-1), dict(max_context_len=-1)):
        assert fn(b=batch(**kw)) == INVALID, kw
    assert fn(H=0) == INVALID and fn(H=3) == INVALID  # not a multiple of the KV heads
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert fn(scale=scale) == INVALID, scale
    assert fn(window=-1) == INVALID
    assert fn(qt=8) == MISALIGNED and fn(qh=24) == MISALIGNED
    assert fn(qt=-16) == INVALID
    one = batch(num_tokens=4)
    assert fn(b=one, q=None) == INVALID
    assert fn(b=one, q=P + 8) == MISALIGNED
    assert fn(b=one, c=cache(base=None)) == INVALID
    assert fn(b=one, c=cache(base=P + 8)) == MISALIGNED
    for f in ("block_table", "q_offsets", "context_lens"):
        assert fn(b=batch(num_tokens=4, **{f: None})) == INVALID, f
    # empty work never reaches the device
    assert fn(b=batch(num_tokens=0), q=None) == OK
    assert fn(b=batch(num_tokens=4, num_reqs=0), q=None) == OK


def test_attention_outputs_refused():
    one = batch(num_tokens=4)
    assert attend(b=one, out=None) == INVALID and attend(b=one, out=P + 8) == MISALIGNED
    assert attend(b=one, ot=2056) == MISALIGNED and attend(b=one, oh=-16) == INVALID
    assert attend(b=one, ws=P + 8, wsb=64) == MISALIGNED and attend(b=one, wsb=-1) == INVALID
    assert mass(b=one, lse=None) == INVALID and mass(b=one, m=None) == INVALID
    assert mass(b=one, w=-1) == INVALID and mass(b=one, rs=-1) == INVALID
    assert mass(b=one, w=0, m=None) == OK


def test_workspace_sizes():
    def size(c=None, H=4, **kw):
        c = cache() if c is None else c
        b = batch(**kw)
        return K._F["kvx_paged_attention_workspace"](ctypes.byref(c), ctypes.byref(b), H)
    assert size(num_tokens=0) == 0
    assert size(num_tokens=3) >= 0
    assert size(c=cache(head_dim=20), num_tokens=3) == -1 and size(H=3, num_tokens=3) == -1
    assert size(num_tokens=-1) == -1


def rope(c=None, q=P, H=4, k=P, v=P, T=5, pos=P, axes=2, axis=None, freq=P, rot=64, slots=P, out=P, qt=2048, kt=512,
         oh=256):
    c = cache() if c is None else c
    axis = [0, 1] * 64 if axis is None else axis
    arr = (ctypes.c_int32 * len(axis))(*axis) if axis != "null" else None
    return K._F["kvx_rope_and_cache"](ctypes.byref(c), q, qt, 256, H, k, kt, 256, v, 512, 256, T, pos, axes, arr, freq, rot, 0,
                                      slots, out, 2048, oh, None, None)


def test_rope_refusals():
    for kw in BAD_CACHES:
        assert rope(c=cache(**kw)) == INVALID, kw
    for kw in ODD_CACHES:
        assert rope(c=cache(**kw), rot=16) == MISALIGNED, kw
    for rot in (0, 8, 24, 144, -16):
        assert rope(rot=rot) == INVALID, rot
    for axes in (0, 5, -1):
        assert rope(axes=axes) == INVALID, axes
    assert rope(axis=[2] * 64) == INVALID and rope(axis=[-1] * 64) == INVALID and rope(axis="null") == INVALID
    assert rope(T=-1) == INVALID and rope(T=1 << 22) == INVALID and rope(H=-1) == INVALID
    for kw in (dict(q=None), dict(out=None), dict(k=None), dict(v=None), dict(pos=None), dict(freq=None), dict(slots=None)):
        assert rope(**kw) == INVALID, kw
    for kw in (dict(q=P + 8), dict(k=P + 2), dict(v=P + 4), dict(out=P + 8), dict(qt=2056), dict(kt=520), dict(oh=8)):
        assert rope(**kw) == MISALIGNED, kw
    assert rope(T=0, q=None, k=None) == OK


def select(m=P, w=500, R=3, H=2, lens=P, budget=100, sink=4, recent=10, keep=P, new=2 * P):
    return K._F["kvx_evict_select"](m, 1000, 500, w, R, H, lens, budget, sink, recent, keep, new, None, None)


def test_select_refusals():
    for kw in (dict(R=-1), dict(R=1 << 21), dict(H=0), dict(w=-1), dict(budget=0), dict(budget=1 << 31), dict(sink=-1), dict(recent=-1),
               dict(sink=101), dict(sink=50, recent=51), dict(m=None), dict(lens=None), dict(keep=None), dict(new=None),
               dict(new=P)):
        assert select(**kw) == INVALID, kw
    assert select(R=0, m=None) == OK


def compact(c=None, src=P, dst=2 * P, cols=8, row=8, dcols=8, drow=8, R=3, H=2, keep=P, budget=100, m=None, mo=None, ms=500,
            mos=500, w=500, wo=500):
    c = cache() if c is None else c
    return K._F["kvx_evict_compact"](ctypes.byref(c), src, cols, row, dst, dcols, drow, R, H, keep, budget, m, 1000, ms, w, mo,
                                     1000, mos, wo, None, None)


def test_compact_refusals():
    for kw in BAD_CACHES:
        assert compact(c=cache(**kw)) == INVALID, kw
    for kw in ODD_CACHES:
        assert compact(c=cache(**kw)) == MISALIGNED, kw
    for kw in (dict(R=-1), dict(R=1 << 20), dict(H=0), dict(H=3), dict(budget=0), dict(cols=9), dict(drow=7), dict(src=None), dict(dst=None),
               dict(keep=None), dict(m=P), dict(mo=P), dict(m=P, mo=2 * P, w=-1), dict(m=P, mo=2 * P, wo=-1),
               dict(m=P, mo=P),  # onto itself, but not in place
               dict(dst=P, m=P, mo=P, mos=400), dict(dst=P, dcols=7), dict(c=cache(base=None)),
               dict(c=cache(num_blocks=0)), dict(cols=0), dict(dcols=0)):
        assert compact(**kw) == INVALID, kw
    assert compact(c=cache(base=P + 8)) == MISALIGNED
    assert compact(R=0, src=None) == OK


def test_binding_refuses_what_the_abi_cannot_see():
    kv = torch.zeros(10, 16, 2, 2, 64, dtype=torch.bfloat16)
    q = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(3, 3, dtype=torch.int32), torch.zeros(3, dtype=torch.int64)
    off = torch.zeros(4, dtype=torch.int64)
    out, lse, m = torch.zeros_like(q), torch.zeros(5, 4), torch.zeros(3, 2, 48)

    def att(**kw):
        a = dict(query=q, kv_cache=kv, block_table=table, q_offsets=off, context_lens=lens, out=out, lse=lse)
        a.update(kw)
        K.kvx_paged_attention(**a)

    for err, kw in [(TypeError, dict(kv_cache=kv.float())), (TypeError, dict(query=q.half(), out=out.half())),
                    (ValueError, dict(kv_cache=kv[0])), (ValueError, dict(layout="blocks_kv_tokens")),
                    (ValueError, dict(query=q[:, :3])), (ValueError, dict(query=q[..., :32])),
                    (ValueError, dict(out=out[:4])), (ValueError, dict(lse=lse[:4])), (TypeError, dict(lse=lse.half())),
                    (ValueError, dict(block_table=table[:2])), (ValueError, dict(block_table=table.long())),
                    (ValueError, dict(q_offsets=off[:3])), (TypeError, dict(context_lens=lens.int())),
                    (ValueError, dict(query=torch.zeros(5, 4, 128, dtype=torch.bfloat16)[..., ::2])),
                    (ValueError, {})]:  # the last: everything fits, but nothing is on a GPU
        with pytest.raises(err):
            att(**kw)
    with pytest.raises(ValueError, match="mass"):
        K.kvx_attention_mass(q, kv, table, off, lens, lse, m[:, :1])
    with pytest.raises(TypeError):
        K.kvx_attention_mass(q, kv, table, off, lens, lse, m.double())
    keep, new = torch.zeros(3, 2, 8, dtype=torch.int32), torch.zeros(3, dtype=torch.int64)
    for kw in (dict(budget=9), dict(keep=keep[:, :1]), dict(new_lens=new[:2]), dict()):
        a = dict(mass=m, context_lens=lens, budget=8, sink=1, recent=1, keep=keep, new_lens=new)
        a.update(kw)
        with pytest.raises(ValueError):
            K.kvx_evict_select(**a)
    for kw in (dict(mass=m), dict(keep=keep[:2]), dict(dst_block_table=table[:2]), dict(keep=keep[:, :0]), dict()):
        a = dict(kv_cache=kv, block_table=table, dst_block_table=table, keep=keep)
        a.update(kw)
        with pytest.raises(ValueError):
            K.kvx_evict_compact(**a)
    k = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    pos, freq, slots = torch.zeros(2, 5, dtype=torch.int64), torch.zeros(32), torch.zeros(5, dtype=torch.int64)
    for kw in (dict(pair_axis=[0] * 31), dict(positions=pos[:, :4].contiguous()), dict(query_out=None), dict(key=q),
               dict(query_out=out[:, :2]), dict()):
        a = dict(query=q, key=k, value=k, positions=pos, inv_freq=freq, pair_axis=[0] * 32, slot_mapping=slots, kv_cache=kv,
                 query_out=out)
        a.update(kw)
        with pytest.raises(ValueError):
            K.kvx_rope_and_cache(**a)


def test_row_counts_past_what_a_launch_can_number():
    """Query rows near 2^31 are refused before anything is enqueued: the kernels count rows of a tile past the last one in
    32 bits, and a launch has at most 2^32 threads."""
    def size(c=None, H=4, **kw):
        c = cache() if c is None else c
        return K._F["kvx_paged_attention_workspace"](ctypes.byref(c), ctypes.byref(batch(**kw)), H)
    one = cache(num_kv_heads=1)
    top = (1 << 31) - 65537  # rows
    for fn in (attend, mass):
        assert fn(c=one, H=1, b=batch(num_tokens=top + 1)) == INVALID
        assert fn(c=one, H=1, b=batch(num_tokens=(1 << 31) - 1)) == INVALID
        assert fn(H=4, b=batch(num_tokens=top // 4 + 1)) == INVALID
        # a count that is taken gets as far as the missing query
        assert fn(c=one, H=1, b=batch(num_tokens=top - 3 * 128), q=None) == INVALID
    assert size(c=one, H=1, num_tokens=top + 1) == -1 and size(c=one, H=1, num_tokens=top - 3 * 128) >= 0
    # a request takes a tile of its own at least: 128 rows for every KV head of it
    many = dict(num_reqs=65535, bt_row_stride=8)
    assert size(c=cache(num_kv_heads=64), H=64, num_tokens=(top - 128 * 64 * 65535) // 64, **many) >= 0
    assert size(c=cache(num_kv_heads=64), H=64, num_tokens=(top - 128 * 64 * 65535) // 64 + 2, **many) == -1
    assert attend(c=cache(num_kv_heads=64), H=64, b=batch(num_tokens=(top - 128 * 64 * 65535) // 64 + 2, **many)) == INVALID
