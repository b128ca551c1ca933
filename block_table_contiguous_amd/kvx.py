"""Python binding of libkvx (include/kvx.h, include/kvx_attention.h): argument marshalling only.

Each kvx_* function here takes torch tensors, checks that they are device tensors of the
right dtype and contiguity, and passes their data pointers, sizes and the current HIP stream
to the C entry point of the same name. Every step of the path runs in libkvx's kernels; there
is no fallback. A non-zero status raises KvxError with the library's status string.

The library is located like the pages' NCCL loader (page "0. vllm 如何使用 nccl 传输 kv cache",
§2.1 and §2.2): an environment variable (KVX_SO_PATH) names it, else the in-tree build is
used; it is opened with ctypes.CDLL and every exported function gets a restype/argtypes
entry from one signature table.
"""
from __future__ import annotations

import ctypes
import os
from array import array
from typing import List, Optional, Sequence

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
DEFAULT_LIB = os.path.join(_HERE, "libkvx.so")

KVX_SUCCESS = 0
KVX_ERR_INVALID_ARGUMENT = 1
KVX_ERR_MISALIGNED = 2
KVX_ERR_CAPACITY = 3
KVX_ERR_HIP = 4

DEVERR_BLOCK_RANGE = 1
DEVERR_TABLE_RANGE = 2
DEVERR_SLOT_RANGE = 4
DEVERR_OFFSETS = 8
DEVERR_TIMEOUT = 16

MODE_PACK, MODE_UNPACK, MODE_DIRECT = 0, 1, 2
MAX_SOURCES = 8
ARRIVALS_BYTES = 4096  # workspace of one signalling copy (KVX_ARRIVALS_BYTES)
NOALLOC_SLOTS = 16  # arrivals workspaces the library keeps per GPU for kvx_pack_signal_noalloc
MAX_EXTENT_BYTES = 1 << 56  # largest byte extent one call may describe (KVX_MAX_EXTENT_BYTES)
XFER_BYTES = 32  # sizeof(kvx_xfer)

DTYPE_BF16, DTYPE_FP16 = 0, 1  # element types of the calls that compute (KVX_DTYPE_*)
MAX_HEAD_DIM = 256
MAX_AXES = 4

_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64



class PagedCache(ctypes.Structure):
    """kvx_paged_cache: one layer's cache for the calls of kvx_attention.h (see paged_cache)."""

    _fields_ = [("base", _P), ("num_blocks", _I64), ("block_stride_bytes", _I64), ("token_stride_bytes", _I64),
                ("kv_stride_bytes", _I64), ("head_stride_bytes", _I64), ("block_size", _I32), ("num_kv_heads", _I32),
                ("head_dim", _I32), ("dtype", _I32)]
    tensor = None  # the tensor that it describes


class Batch(ctypes.Structure):
    """kvx_batch: the requests of one attention call."""

    _fields_ = [("block_table", _P), ("q_offsets", _P), ("context_lens", _P), ("max_blocks_per_req", _I64),
                ("bt_row_stride", _I64), ("num_tokens", _I64), ("max_query_len", _I64), ("max_context_len", _I64),
                ("num_reqs", _I32)]


_F32 = ctypes.c_float
_CACHE, _BATCH = ctypes.POINTER(PagedCache), ctypes.POINTER(Batch)

# name -> (restype, argtypes); mirrors include/kvx.h and include/kvx_attention.h
SIGNATURES = {
    "kvx_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "kvx_abi_version": (_I32, []),
    "kvx_slot_mapping": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _P, _I64, _I32, _P, _P, _P]),
    "kvx_reshape_and_cache": (ctypes.c_int, [_P, _I64, _P, _I64, _I64, _I64, _P, _P, _I64, _I32,
                                             _I64, _I64, _I64, _P, _P]),
    "kvx_build_xfer_list": (ctypes.c_int, [_P, _P, _P, _I32, _I64, _I32, _P, _I64, _P, _P, _P]),
    "kvx_pack": (ctypes.c_int, [_P, _I32, _I64, _I64, _P, _P, _I64, _P, _P, _P]),
    "kvx_unpack": (ctypes.c_int, [_P, _I32, _P, _I32, _I64, _I64, _I32, _P, _P, _I64, _P, _P]),
    "kvx_pack_split": (ctypes.c_int, [_P, _I32, _I64, _I64, _I32, _P, _P, _I64, _P, _I32, _P, _P]),
    "kvx_pack_kv_first": (ctypes.c_int, [_P, _I32, _I64, _I64, _I64, _P, _I32, _P, _P, _I64, _P, _P, _P]),
    "kvx_unpack_kv_first": (ctypes.c_int, [_P, _P, _I32, _I64, _I64, _I64, _P, _I32, _P, _P, _I64, _P, _P]),
    "kvx_copy_direct": (ctypes.c_int, [_P, _P, _I32, _I64, _I64, _I64, _P, _P, _I64, _P, _P]),
    "kvx_signal_add": (ctypes.c_int, [_P, ctypes.c_uint64, _P]),
    "kvx_signal_wait": (ctypes.c_int, [_P, ctypes.c_uint64, _I64, _P, _P]),
    "kvx_pack_signal": (ctypes.c_int, [_P, _I32, _I64, _I64, _P, _P, _I64, _P, _P, ctypes.c_uint64, _P, _P, _P]),
    "kvx_copy_direct_signal": (ctypes.c_int, [_P, _P, _I32, _I64, _I64, _I64, _P, _P, _I64, _P, ctypes.c_uint64,
                                              _P, _P, _P]),
    "kvx_pack_signal_noalloc": (ctypes.c_int, [_P, _I32, _I64, _I64, _P, _P, _I64, _P, _P, ctypes.c_uint64, _I32,
                                               _P, _P]),
    "kvx_rope_and_cache": (ctypes.c_int, [_CACHE, _P, _I64, _I64, _I32, _P, _I64, _I64, _P, _I64, _I64, _I64, _P, _I32,
                                          _P, _P, _I32, _I32, _P, _P, _I64, _I64, _P, _P]),
    "kvx_paged_attention": (ctypes.c_int, [_CACHE, _BATCH, _P, _I64, _I64, _I32, _F32, _I32, _I64, _P, _I64, _I64, _P,
                                           _P, _I64, _P, _P]),
    "kvx_paged_attention_workspace": (_I64, [_CACHE, _BATCH, _I32]),
    "kvx_attention_mass": (ctypes.c_int, [_CACHE, _BATCH, _P, _I64, _I64, _I32, _F32, _I32, _I64, _P, _P, _I64, _I64,
                                          _I64, _P, _P]),
    "kvx_evict_select": (ctypes.c_int, [_P, _I64, _I64, _I64, _I32, _I32, _P, _I64, _I64, _I64, _P, _P, _P, _P]),
    "kvx_evict_compact": (ctypes.c_int, [_CACHE, _P, _I64, _I64, _P, _I64, _I64, _I32, _I32, _P, _I64, _P, _I64, _I64,
                                         _I64, _P, _I64, _I64, _I64, _P, _P]),
}


class KvxError(RuntimeError):
    def __init__(self, fn: str, status: int, message: str):
        super().__init__(f"{fn}: {message} (status {status})")
        self.status = status


def library_path() -> str:
    return os.environ.get("KVX_SO_PATH") or DEFAULT_LIB


def _load():
    path = library_path()
    if not os.path.exists(path):
        raise ImportError(
            f"libkvx not found at {path}: build it with `python -m block_table_contiguous_amd.build` "
            "(the KV transfer path has no fallback)")
    lib = ctypes.CDLL(path)
    funcs = {}
    for name, (restype, argtypes) in SIGNATURES.items():
        f = getattr(lib, name)
        f.restype = restype
        f.argtypes = argtypes
        funcs[name] = f
    return lib, funcs


LIB, _F = _load()


def kvx_status_string(status: int) -> str:
    return _F["kvx_status_string"](int(status)).decode()


def kvx_abi_version() -> int:
    return int(_F["kvx_abi_version"]())


def _check(fn: str, status: int):
    if status != KVX_SUCCESS:
        raise KvxError(fn, status, kvx_status_string(status))


# ---------------------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------------------

def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("kvx: tensors must live on the GPU")
    return t.data_ptr()


_raw_stream = None  # torch's internal raw-handle query, once it has been seen to agree


def _public_stream() -> int:
    import torch

    return torch.cuda.current_stream().cuda_stream


def _current_stream() -> int:
    """The current device's current stream handle. torch.cuda.current_stream() builds a Stream
    object per call (a third of a small call's host time), so the binding uses torch's raw
    handle query instead, but only after checking once that it returns the same handle as the
    public API; if the query is missing or disagrees, every call uses the public API."""
    global _raw_stream
    if _raw_stream is None:
        import torch

        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        dev = getattr(torch._C, "_cuda_getDevice", None)
        fast = None
        if raw is not None and dev is not None:
            fast = lambda: raw(dev())  # noqa: E731
            try:
                if fast() != _public_stream():
                    fast = None
            except Exception:  # a changed signature: fall back to the public API
                fast = None
        _raw_stream = fast or _public_stream
    return _raw_stream()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return _current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _rows_contiguous(t) -> bool:
    """Every t[i] is densely packed (the dimensions after the first are contiguous)."""
    if t.is_contiguous():  # the common case, without walking the strides
        return True
    expect = 1
    for size, stride in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if size != 1 and stride != expect:
            return False
        expect *= size
    return True


def _want(t, dtype, name):
    if t.dtype != dtype:
        raise TypeError(f"kvx: {name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"kvx: {name} must be contiguous")


def _want_runs(xfers, xfer_count, total_blocks: int):
    """A run list the copy kernels may read up to total_blocks records of."""
    import torch

    _want(xfers, torch.int64, "xfers")
    _want(xfer_count, torch.int64, "xfer_count")
    if xfers.numel() // 4 < total_blocks or xfer_count.numel() < 1:
        raise ValueError("kvx: the run list holds fewer than total_blocks records")


def layer_base_table(layers: Sequence, device=None):
    """Device int64 array of the layers' base addresses (the per-layer cache pointers the
    pack/unpack kernels index)."""
    import torch

    dev = device if device is not None else layers[0].device
    return torch.tensor([t.data_ptr() for t in layers], dtype=torch.int64, device=dev)


def flatten_tables(tables: Sequence[np.ndarray], device):
    """Per-request id lists -> (ids int32 [N], req_offsets int64 [R+1]) device tensors (CSR)."""
    import torch

    counts = np.array([len(t) for t in tables], dtype=np.int64)
    offsets = np.zeros(len(tables) + 1, dtype=np.int64)
    np.cumsum(counts, out=offsets[1:])
    ids = np.concatenate([np.asarray(t, np.int32) for t in tables]) if len(tables) else np.zeros(0, np.int32)
    return (torch.from_numpy(np.ascontiguousarray(ids, np.int32)).to(device),
            torch.from_numpy(offsets).to(device))


def new_xfer_list(capacity: int, device):
    """Storage for `capacity` kvx_xfer records (int64 [capacity][4]) plus its count."""
    import torch

    return (torch.zeros((max(int(capacity), 1), 4), dtype=torch.int64, device=device),
            torch.zeros(1, dtype=torch.int64, device=device))


def decode_xfers(xfers, count) -> List[tuple]:
    """Host copy of a run list as (src_block, dst_block, buf_block, num_blocks, req) tuples."""
    n = int(count.item()) if hasattr(count, "item") else int(count)
    raw = xfers[:n].cpu().numpy()
    tail = raw[:, 3].copy().view(np.int32).reshape(n, 2)
    return [(int(a), int(b), int(c), int(t[0]), int(t[1])) for (a, b, c, _), t in zip(raw, tail)]


def cache_strides(kv_cache, layout: str = "blocks_tokens_kv"):
    """(num_blocks, block_size, block_stride, token_stride, kv_stride) in bytes for a 5-D cache
    tensor in one of three layouts:
      blocks_tokens_kv  [blocks][block_size][K,V][heads][head_dim]
      blocks_kv_tokens  [blocks][K,V][block_size][heads][head_dim]
      kv_blocks_tokens  [K,V][blocks][block_size][heads][head_dim]"""
    e = kv_cache.element_size()
    s = [x * e for x in kv_cache.stride()]
    sh = kv_cache.shape
    if layout == "blocks_tokens_kv":
        return sh[0], sh[1], s[0], s[1], s[2]
    if layout == "blocks_kv_tokens":
        return sh[0], sh[2], s[0], s[2], s[1]
    if layout == "kv_blocks_tokens":
        return sh[1], sh[2], s[1], s[2], s[0]
    raise ValueError(f"unknown layout {layout}")


# ---------------------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ---------------------------------------------------------------------------------------

def kvx_slot_mapping(block_table, req_idx, positions, block_size: int, slot_mapping,
                     err_flag=None, max_blocks_per_req: Optional[int] = None, stream=None):
    """slot_mapping[i] = block_table[req_idx[i], positions[i] // bs] * bs + positions[i] % bs."""
    import torch

    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.stride(1) != 1:
        raise ValueError("kvx: block_table must be a row-major int32 [num_reqs][width] tensor")
    _want(req_idx, torch.int32, "req_idx")
    _want(positions, torch.int64, "positions")
    _want(slot_mapping, torch.int64, "slot_mapping")
    T = req_idx.numel()
    if positions.numel() != T or slot_mapping.numel() != T:
        raise ValueError("kvx: req_idx, positions and slot_mapping need the same length")
    width = block_table.shape[1] if max_blocks_per_req is None else int(max_blocks_per_req)
    if width > block_table.shape[1]:
        raise ValueError("kvx: max_blocks_per_req is wider than the block table")
    # a one-row table's row stride is never used (it can be 0 for a broadcast row)
    row_stride = block_table.stride(0) if block_table.shape[0] > 1 else max(block_table.shape[1], width)
    st = _F["kvx_slot_mapping"](_ptr(block_table), block_table.shape[0], width,
                                row_stride, _ptr(req_idx), _ptr(positions), T,
                                int(block_size), _ptr(slot_mapping), _ptr(err_flag), _stream(stream))
    _check("kvx_slot_mapping", st)


def kvx_reshape_and_cache(key, value, slot_mapping, kv_cache, num_blocks: int, block_size: int,
                          block_stride_bytes: int, token_stride_bytes: int, kv_stride_bytes: int,
                          err_flag=None, stream=None):
    """Write key[i] / value[i] rows into kv_cache at slot_mapping[i] (negative slot = skip)."""
    import torch

    _want(slot_mapping, torch.int64, "slot_mapping")
    T = slot_mapping.numel()
    if key.shape[0] != T or value.shape[0] != T or key.shape != value.shape:
        raise ValueError("kvx: key/value must be [num_tokens, ...] of the same shape")
    e = key.element_size()
    row = key.numel() // T * e if T else 0
    for name, t in (("key", key), ("value", value)):
        if not _rows_contiguous(t):
            raise ValueError(f"kvx: each {name} row must be contiguous")
    if T and num_blocks > 0:
        last = ((int(num_blocks) - 1) * int(block_stride_bytes) + (int(block_size) - 1) * int(token_stride_bytes)
                + int(kv_stride_bytes) + row)
        room = kv_cache.untyped_storage().nbytes() - kv_cache.storage_offset() * kv_cache.element_size()
        if last > room:
            raise ValueError("kvx: num_blocks, block_size and the strides address bytes past the end of kv_cache")
    st = _F["kvx_reshape_and_cache"](_ptr(key), key.stride(0) * e, _ptr(value), value.stride(0) * e,
                                     T, row, _ptr(slot_mapping), _ptr(kv_cache), int(num_blocks),
                                     int(block_size), int(block_stride_bytes), int(token_stride_bytes),
                                     int(kv_stride_bytes), _ptr(err_flag), _stream(stream))
    _check("kvx_reshape_and_cache", st)


def kvx_build_xfer_list(src_ids, dst_ids, req_offsets, mode: int, xfers, xfer_count,
                        err_flag=None, stream=None):
    """Cut the CSR block lists into maximal runs (see include/kvx.h)."""
    import torch

    _want(req_offsets, torch.int64, "req_offsets")
    for name, t in (("src_ids", src_ids), ("dst_ids", dst_ids)):
        if t is not None:
            _want(t, torch.int32, name)
    _want(xfers, torch.int64, "xfers")
    if req_offsets.numel() < 1:
        raise ValueError("kvx: req_offsets needs num_reqs + 1 entries")
    if src_ids is not None and dst_ids is not None and src_ids.numel() != dst_ids.numel():
        raise ValueError("kvx: src_ids and dst_ids must list the same number of blocks")
    ref = src_ids if src_ids is not None else dst_ids
    total = ref.numel() if ref is not None else 0
    capacity = xfers.numel() // 4
    st = _F["kvx_build_xfer_list"](_ptr(src_ids), _ptr(dst_ids), _ptr(req_offsets),
                                   req_offsets.numel() - 1, total, int(mode), _ptr(xfers), capacity,
                                   _ptr(xfer_count), _ptr(err_flag), _stream(stream))
    _check("kvx_build_xfer_list", st)


def kvx_pack(layer_bases, block_bytes: int, num_cache_blocks: int, xfers, xfer_count,
             total_blocks: int, send_buf, err_flag=None, stream=None):
    """Gather the listed blocks of every layer into send_buf [L][total_blocks][block_bytes]."""
    import torch

    _want(layer_bases, torch.int64, "layer_bases")
    _want_runs(xfers, xfer_count, total_blocks)
    L = layer_bases.numel()
    if send_buf.numel() * send_buf.element_size() < L * total_blocks * block_bytes:
        raise ValueError("kvx: send_buf smaller than num_layers * total_blocks * block_bytes")
    st = _F["kvx_pack"](_ptr(layer_bases), L, int(block_bytes), int(num_cache_blocks), _ptr(xfers),
                        _ptr(xfer_count), int(total_blocks), _ptr(send_buf), _ptr(err_flag),
                        _stream(stream))
    _check("kvx_pack", st)


def kvx_unpack(send_bufs: Sequence, layer_bases, block_bytes: int, num_cache_blocks: int,
               rows_per_block: int, xfers, xfer_count, total_blocks: int, err_flag=None,
               stream=None):
    """Scatter send buffer(s) into the listed destination blocks; with several sources each
    destination row is the concatenation of the sources' rows (head merge)."""
    import torch

    _want(layer_bases, torch.int64, "layer_bases")
    _want_runs(xfers, xfer_count, total_blocks)
    L = layer_bases.numel()
    S = len(send_bufs)
    if not 1 <= S <= MAX_SOURCES:
        raise ValueError(f"kvx: 1..{MAX_SOURCES} send buffers")
    for b in send_bufs:
        if b.numel() * b.element_size() < L * total_blocks * (block_bytes // S):
            raise ValueError("kvx: a send buffer is smaller than num_layers * total_blocks * block_bytes/num_src")
    arr = (ctypes.c_void_p * S)(*[_ptr(b) for b in send_bufs])
    st = _F["kvx_unpack"](arr, S, _ptr(layer_bases), L, int(block_bytes), int(num_cache_blocks),
                          int(rows_per_block), _ptr(xfers), _ptr(xfer_count), int(total_blocks),
                          _ptr(err_flag), _stream(stream))
    _check("kvx_unpack", st)


def kvx_copy_direct(src_layer_bases, dst_layer_bases, block_bytes: int, src_num_blocks: int,
                    dst_num_blocks: int, xfers, xfer_count, total_blocks: int, err_flag=None,
                    stream=None):
    """Copy the listed blocks of every layer from the source caches straight into the
    destination caches (no buffer); the runs come from kvx_build_xfer_list(MODE_DIRECT)."""
    import torch

    _want(src_layer_bases, torch.int64, "src_layer_bases")
    _want(dst_layer_bases, torch.int64, "dst_layer_bases")
    _want_runs(xfers, xfer_count, total_blocks)
    L = src_layer_bases.numel()
    if dst_layer_bases.numel() != L:
        raise ValueError("kvx: source and destination layer tables differ in length")
    st = _F["kvx_copy_direct"](_ptr(src_layer_bases), _ptr(dst_layer_bases), L, int(block_bytes),
                               int(src_num_blocks), int(dst_num_blocks), _ptr(xfers), _ptr(xfer_count),
                               int(total_blocks), _ptr(err_flag), _stream(stream))
    _check("kvx_copy_direct", st)


def kvx_pack_split(layer_bases, block_bytes: int, num_cache_blocks: int, rows_per_block: int,
                   xfers, xfer_count, total_blocks: int, send_bufs: Sequence, err_flag=None,
                   stream=None):
    """Pack for num_dst receivers that each own a head shard: send_bufs[d] gets piece d of
    every row of every listed block (the inverse of kvx_unpack's merge)."""
    import torch

    _want(layer_bases, torch.int64, "layer_bases")
    _want_runs(xfers, xfer_count, total_blocks)
    L = layer_bases.numel()
    D = len(send_bufs)
    if not 1 <= D <= MAX_SOURCES:
        raise ValueError(f"kvx: 1..{MAX_SOURCES} send buffers")
    for b in send_bufs:
        if b.numel() * b.element_size() < L * total_blocks * (block_bytes // D):
            raise ValueError("kvx: a send buffer is smaller than num_layers * total_blocks * block_bytes/num_dst")
    arr = (ctypes.c_void_p * D)(*[_ptr(b) for b in send_bufs])
    st = _F["kvx_pack_split"](_ptr(layer_bases), L, int(block_bytes), int(num_cache_blocks),
                              int(rows_per_block), _ptr(xfers), _ptr(xfer_count), int(total_blocks), arr, D,
                              _ptr(err_flag), _stream(stream))
    _check("kvx_pack_split", st)


def kvx_pack_kv_first(layer_bases, segment_bytes: int, plane_stride_bytes: int, num_cache_blocks: int,
                      req_offsets, xfers, xfer_count, total_blocks: int, send_buf, err_flag=None,
                      stream=None):
    """Pack from kv-first caches: per layer and request, the K segments then the V segments."""
    import torch

    _want(layer_bases, torch.int64, "layer_bases")
    _want_runs(xfers, xfer_count, total_blocks)
    _want(req_offsets, torch.int64, "req_offsets")
    L = layer_bases.numel()
    if send_buf.numel() * send_buf.element_size() < L * 2 * total_blocks * segment_bytes:
        raise ValueError("kvx: send_buf smaller than num_layers * 2 * total_blocks * segment_bytes")
    st = _F["kvx_pack_kv_first"](_ptr(layer_bases), L, int(segment_bytes), int(plane_stride_bytes),
                                 int(num_cache_blocks), _ptr(req_offsets), req_offsets.numel() - 1,
                                 _ptr(xfers), _ptr(xfer_count), int(total_blocks), _ptr(send_buf),
                                 _ptr(err_flag), _stream(stream))
    _check("kvx_pack_kv_first", st)


def kvx_unpack_kv_first(send_buf, layer_bases, segment_bytes: int, plane_stride_bytes: int,
                        num_cache_blocks: int, req_offsets, xfers, xfer_count, total_blocks: int,
                        err_flag=None, stream=None):
    """Scatter a kv-first buffer (per request: K segments, then V segments) into kv-first caches."""
    import torch

    _want(layer_bases, torch.int64, "layer_bases")
    _want_runs(xfers, xfer_count, total_blocks)
    _want(req_offsets, torch.int64, "req_offsets")
    L = layer_bases.numel()
    if send_buf.numel() * send_buf.element_size() < L * 2 * total_blocks * segment_bytes:
        raise ValueError("kvx: send_buf smaller than num_layers * 2 * total_blocks * segment_bytes")
    st = _F["kvx_unpack_kv_first"](_ptr(send_buf), _ptr(layer_bases), L, int(segment_bytes),
                                   int(plane_stride_bytes), int(num_cache_blocks), _ptr(req_offsets),
                                   req_offsets.numel() - 1, _ptr(xfers), _ptr(xfer_count), int(total_blocks),
                                   _ptr(err_flag), _stream(stream))
    _check("kvx_unpack_kv_first", st)


def new_arrivals(device):
    """A zeroed arrivals workspace for the signalling copies (one per concurrent stream)."""
    import torch

    return torch.zeros(ARRIVALS_BYTES // 4, dtype=torch.int32, device=device)


def _want_signal(counter, arrivals):
    import torch

    _want(counter, torch.int64, "counter")
    _want(arrivals, torch.int32, "arrivals")
    if counter.numel() < 1 or arrivals.numel() * 4 < ARRIVALS_BYTES:
        raise ValueError(f"kvx: counter needs one element and arrivals {ARRIVALS_BYTES} bytes")


def kvx_pack_signal(layer_bases, block_bytes: int, num_cache_blocks: int, xfers, xfer_count,
                    total_blocks: int, send_buf, counter, arrivals, delta: int = 1, err_flag=None,
                    stream=None):
    """kvx_pack whose launch also adds `delta` to `counter` (int64 device tensor, read as
    uint64) once every packed byte is visible device-wide. `arrivals` is an int32 device
    tensor of ARRIVALS_BYTES // 4 zeros (new_arrivals); each call leaves it all zero again
    (one per concurrent stream)."""
    import torch

    _want(layer_bases, torch.int64, "layer_bases")
    _want_runs(xfers, xfer_count, total_blocks)
    _want_signal(counter, arrivals)
    L = layer_bases.numel()
    if send_buf.numel() * send_buf.element_size() < L * total_blocks * block_bytes:
        raise ValueError("kvx: send_buf smaller than num_layers * total_blocks * block_bytes")
    st = _F["kvx_pack_signal"](_ptr(layer_bases), L, int(block_bytes), int(num_cache_blocks), _ptr(xfers),
                               _ptr(xfer_count), int(total_blocks), _ptr(send_buf), _ptr(counter), int(delta),
                               _ptr(arrivals), _ptr(err_flag), _stream(stream))
    _check("kvx_pack_signal", st)


def kvx_pack_signal_noalloc(layer_bases, block_bytes: int, num_cache_blocks: int, xfers, xfer_count,
                            total_blocks: int, send_buf, counter, slot: int = 0, delta: int = 1, err_flag=None,
                            stream=None):
    """kvx_pack_signal with the arrivals workspace taken from the library's own static array
    (workspace `slot` of NOALLOC_SLOTS): nothing is allocated, here or in the library. Calls
    that use the same slot must not overlap in time; the stream must belong to the current
    device."""
    import torch

    _want(layer_bases, torch.int64, "layer_bases")
    _want_runs(xfers, xfer_count, total_blocks)
    _want(counter, torch.int64, "counter")
    L = layer_bases.numel()
    if send_buf.numel() * send_buf.element_size() < L * total_blocks * block_bytes:
        raise ValueError("kvx: send_buf smaller than num_layers * total_blocks * block_bytes")
    st = _F["kvx_pack_signal_noalloc"](_ptr(layer_bases), L, int(block_bytes), int(num_cache_blocks), _ptr(xfers),
                                       _ptr(xfer_count), int(total_blocks), _ptr(send_buf), _ptr(counter),
                                       int(delta), int(slot), _ptr(err_flag), _stream(stream))
    _check("kvx_pack_signal_noalloc", st)


def kvx_copy_direct_signal(src_layer_bases, dst_layer_bases, block_bytes: int, src_num_blocks: int,
                           dst_num_blocks: int, xfers, xfer_count, total_blocks: int, counter, arrivals,
                           delta: int = 1, err_flag=None, stream=None):
    """kvx_copy_direct whose launch also adds `delta` to `counter` once every copied byte is
    visible device-wide (the one-sided write with its signal); `arrivals` as kvx_pack_signal."""
    import torch

    _want(src_layer_bases, torch.int64, "src_layer_bases")
    _want(dst_layer_bases, torch.int64, "dst_layer_bases")
    _want_runs(xfers, xfer_count, total_blocks)
    _want_signal(counter, arrivals)
    L = src_layer_bases.numel()
    if dst_layer_bases.numel() != L:
        raise ValueError("kvx: source and destination layer tables differ in length")
    st = _F["kvx_copy_direct_signal"](_ptr(src_layer_bases), _ptr(dst_layer_bases), L, int(block_bytes),
                                      int(src_num_blocks), int(dst_num_blocks), _ptr(xfers), _ptr(xfer_count),
                                      int(total_blocks), _ptr(counter), int(delta), _ptr(arrivals),
                                      _ptr(err_flag), _stream(stream))
    _check("kvx_copy_direct_signal", st)


def kvx_signal_add(counter, delta: int = 1, stream=None):
    """Once the work enqueued on `stream` so far has finished, add `delta` to the uint64
    counter (an int64 device tensor of one element, read as unsigned)."""
    _want(counter, _torch_int64(), "counter")
    _check("kvx_signal_add", _F["kvx_signal_add"](_ptr(counter), int(delta), _stream(stream)))


def kvx_signal_wait(counter, value: int, timeout_us: int = 10_000_000, err=None, stream=None):
    """Hold the work enqueued on `stream` after this call until counter >= value (polled on
    the GPU); after timeout_us the wait ends and sets DEVERR_TIMEOUT in `err`."""
    _want(counter, _torch_int64(), "counter")
    _check("kvx_signal_wait", _F["kvx_signal_wait"](_ptr(counter), int(value), int(timeout_us),
                                                    _ptr(err), _stream(stream)))


def _torch_int64():
    import torch

    return torch.int64


# ---------------------------------------------------------------------------------------
# calls that compute on a paged cache (include/kvx_attention.h)
# ---------------------------------------------------------------------------------------
# A decode step makes a few of these calls a layer, so the checks read each shape and stride once.

_ELEMENTS = {}  # torch element type -> DTYPE_*, filled on first use
_device_query = None  # as _raw_stream: torch's internal query of the current device, if it is there


def _dtype_code(dtype, name: str) -> int:
    if not _ELEMENTS:
        import torch

        _ELEMENTS.update({torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_FP16})
    code = _ELEMENTS.get(dtype)
    if code is None:
        raise TypeError(f"kvx: {name} must be bfloat16 or float16, got {dtype}")
    return code


def _current_device() -> int:
    global _device_query
    if _device_query is None:
        import torch

        query = getattr(torch._C, "_cuda_getDevice", None)
        _device_query = query if query is not None and query() == torch.cuda.current_device() \
            else torch.cuda.current_device
    return _device_query()


def _on_current_device(tensors):
    """Every tensor given lives on the current device, whose stream the call is enqueued on."""
    where = {t.get_device() for t in tensors if t is not None}
    if min(where) < 0:
        raise ValueError("kvx: tensors must live on the GPU")
    if where != {_current_device()}:
        raise ValueError("kvx: every tensor must live on the current device")


def paged_cache(kv_cache, layout: str = "blocks_tokens_kv") -> PagedCache:
    """A 5-D cache tensor (one of cache_strides' layouts, any strides whose last dimension is
    dense) as the struct that the calls below take. They make it from the tensor themselves; a
    caller that makes the same call many times can make it once and pass it instead."""
    shape, stride = kv_cache.shape, kv_cache.stride()
    b, o, w = {"blocks_tokens_kv": (0, 1, 2), "blocks_kv_tokens": (0, 2, 1), "kv_blocks_tokens": (1, 2, 0)}.get(
        layout, (0, 0, 0))
    if b == o:
        raise ValueError(f"unknown layout {layout}")
    if len(shape) != 5 or shape[w] != 2:
        raise ValueError("kvx: kv_cache must be a 5-D cache tensor of the given layout")
    code = _dtype_code(kv_cache.dtype, "kv_cache")
    if shape[4] > 1 and stride[4] != 1:
        raise ValueError("kvx: the last dimension of kv_cache must be dense")
    # the stride of a dimension with one entry is never used and may be anything
    c = PagedCache(kv_cache.data_ptr(), shape[b], 2 * stride[b] if shape[b] > 1 else 0,
                   2 * stride[o] if shape[o] > 1 else 0, 2 * stride[w], 2 * stride[3] if shape[3] > 1 else 0, shape[o],
                   shape[3], shape[4], code)
    c.tensor = kv_cache  # kept alive, and looked at for its device
    return c


def _cache(kv_cache, layout) -> PagedCache:
    return kv_cache if type(kv_cache) is PagedCache else paged_cache(kv_cache, layout)


def _rows(t, tokens: int, heads, cache: PagedCache, name: str):
    """Byte strides (token, head) of a [tokens][heads][head_dim] tensor of the cache's element type,
    its last dimension dense (heads None: any number)."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[0] != tokens or (heads is not None and shape[1] != heads) or shape[2] != cache.head_dim:
        raise ValueError(f"kvx: {name} must be [num_tokens][heads][head_dim]")
    if _dtype_code(t.dtype, name) != cache.dtype:
        raise TypeError(f"kvx: {name} and kv_cache must have the same element type")
    if stride[2] != 1 and shape[2] > 1:
        raise ValueError(f"kvx: the last dimension of {name} must be dense")
    return 2 * stride[0] if shape[0] > 1 else 0, 2 * stride[1] if shape[1] > 1 else 0


def _table(t, reqs: int, name: str = "block_table"):
    """(columns, row stride) of a block table with a row a request."""
    import torch

    shape, stride = t.shape, t.stride()
    if t.dtype != torch.int32 or len(shape) != 2 or (shape[1] > 1 and stride[1] != 1):
        raise ValueError(f"kvx: {name} must be a row-major int32 [num_reqs][width] tensor")
    if shape[0] != reqs:
        raise ValueError(f"kvx: {name} needs a row a request")
    return shape[1], stride[0] if shape[0] > 1 else shape[1]


def _lists(t, name: str, reqs: int, heads: Optional[int]):
    """(request stride, head stride, width) of float32 [num_reqs][heads][width], the last dimension
    dense."""
    import torch

    shape, stride = t.shape, t.stride()
    if t.dtype != torch.float32:
        raise TypeError(f"kvx: {name} must be torch.float32, got {t.dtype}")
    if len(shape) != 3 or shape[0] != reqs or (heads is not None and shape[1] != heads):
        raise ValueError(f"kvx: {name} must be [num_reqs][heads][width]")
    if shape[2] > 1 and stride[2] != 1:
        raise ValueError(f"kvx: the last dimension of {name} must be dense")
    return stride[0] if shape[0] > 1 else 0, stride[1] if shape[1] > 1 else 0, shape[2]


def kvx_rope_and_cache(query, key, value, positions, inv_freq, pair_axis: Sequence[int], slot_mapping, kv_cache,
                       query_out, layout: str = "blocks_tokens_kv", interleaved: bool = False, err_flag=None,
                       stream=None):
    """Rotate query into query_out and key into the cache by positions ([num_axes][num_tokens]),
    pair i by positions[pair_axis[i]] * inv_freq[i], and write the rotated K row and the V row of
    every token through its slot (negative slot = no row). query and query_out may be None."""
    import torch

    c = _cache(kv_cache, layout)
    _want(slot_mapping, torch.int64, "slot_mapping")
    _want(positions, torch.int64, "positions")
    _want(inv_freq, torch.float32, "inv_freq")
    T = slot_mapping.numel()
    axes = positions.shape
    if len(axes) != 2 or axes[1] != T:
        raise ValueError("kvx: positions must be [num_axes][num_tokens]")
    pairs = len(pair_axis)
    if inv_freq.numel() != pairs:
        raise ValueError("kvx: pair_axis and inv_freq need one entry a pair")
    if (query is None) != (query_out is None):
        raise ValueError("kvx: query and query_out go together")
    ks = _rows(key, T, c.num_kv_heads, c, "key")
    vs = _rows(value, T, c.num_kv_heads, c, "value")
    heads, qs, os_, q_ptr, o_ptr = 0, (0, 0), (0, 0), None, None
    if query is not None:
        qs = _rows(query, T, None, c, "query")
        heads = query.shape[1]
        os_ = _rows(query_out, T, heads, c, "query_out")
        q_ptr, o_ptr = query.data_ptr(), query_out.data_ptr()
    _on_current_device((query, key, value, positions, inv_freq, slot_mapping, c.tensor, query_out, err_flag))
    axis_of = array("i", pair_axis if pairs else (0,))  # a ctypes array of as many costs three times this
    st = _F["kvx_rope_and_cache"](
        c, q_ptr, *qs, heads, key.data_ptr(), *ks, value.data_ptr(), *vs, T, positions.data_ptr(), axes[0],
        axis_of.buffer_info()[0], inv_freq.data_ptr(), 2 * pairs, bool(interleaved), slot_mapping.data_ptr(),
        o_ptr, *os_, _ptr(err_flag), _stream(stream))
    _check("kvx_rope_and_cache", st)


def _batch(query, c: PagedCache, block_table, q_offsets, context_lens, max_query_len, max_context_len):
    """(Batch, query heads, query strides)."""
    import torch

    T, heads = query.shape[0], query.shape[1] if query.dim() == 3 else 0
    qs = _rows(query, T, None, c, "query")
    if heads == 0 or heads % c.num_kv_heads:
        raise ValueError("kvx: the query heads must be a multiple of the KV heads")
    _want(q_offsets, torch.int64, "q_offsets")
    _want(context_lens, torch.int64, "context_lens")
    R = context_lens.numel()
    if q_offsets.numel() != R + 1:
        raise ValueError("kvx: q_offsets needs num_reqs + 1 entries")
    width, row = _table(block_table, R)
    # plain addresses: _on_current_device looks at the tensors before the call
    b = Batch(block_table.data_ptr(), q_offsets.data_ptr(), context_lens.data_ptr(), width, row, T,
              T if max_query_len is None else int(max_query_len),
              width * c.block_size if max_context_len is None else int(max_context_len), R)
    return b, heads, qs


def attention_workspace_bytes(query, kv_cache, num_reqs: int, max_query_len: int, max_context_len: int,
                              layout: str = "blocks_tokens_kv") -> int:
    """Bytes of workspace with which kvx_paged_attention splits such a batch as far as pays."""
    c = _cache(kv_cache, layout)
    b = Batch(None, None, None, 0, 0, query.shape[0], int(max_query_len), int(max_context_len), int(num_reqs))
    n = _F["kvx_paged_attention_workspace"](c, b, query.shape[1])
    if n < 0:
        raise ValueError("kvx: kvx_paged_attention does not take a batch of these sizes")
    return int(n)


def new_attention_workspace(query, kv_cache, num_reqs: int, max_query_len: int, max_context_len: int,
                            layout: str = "blocks_tokens_kv"):
    """A workspace of attention_workspace_bytes (one per concurrent stream or captured graph)."""
    import torch

    n = attention_workspace_bytes(query, kv_cache, num_reqs, max_query_len, max_context_len, layout)
    return torch.empty(n, dtype=torch.uint8, device=query.device)


def _want_lse(lse, T: int, heads: int):
    import torch

    _want(lse, torch.float32, "lse")
    if tuple(lse.shape) != (T, heads):
        raise ValueError("kvx: lse must be [num_tokens][heads]")


def kvx_paged_attention(query, kv_cache, block_table, q_offsets, context_lens, out, lse=None,
                        scale: Optional[float] = None, causal: bool = True, window: int = 0,
                        max_query_len: Optional[int] = None, max_context_len: Optional[int] = None, workspace=None,
                        layout: str = "blocks_tokens_kv", err_flag=None, stream=None):
    """Attention of each request's new tokens (rows q_offsets[r] .. q_offsets[r+1]-1 of query,
    [num_tokens][heads][head_dim]) over its paged cache of context_lens[r] slots, into out and,
    if given, lse (float32 [num_tokens][heads]). scale defaults to head_dim ** -0.5; max_query_len
    and max_context_len only choose the launch shape."""
    c = _cache(kv_cache, layout)
    b, heads, qs = _batch(query, c, block_table, q_offsets, context_lens, max_query_len, max_context_len)
    os_ = _rows(out, b.num_tokens, heads, c, "out")
    if lse is not None:
        _want_lse(lse, b.num_tokens, heads)
    nbytes = 0
    if workspace is not None:
        if not workspace.is_contiguous():
            raise ValueError("kvx: workspace must be contiguous")
        nbytes = workspace.numel() * workspace.element_size()
    _on_current_device((query, c.tensor, block_table, q_offsets, context_lens, out, lse, workspace, err_flag))
    st = _F["kvx_paged_attention"](
        c, b, query.data_ptr(), *qs, heads, c.head_dim ** -0.5 if scale is None else float(scale), bool(causal), int(window),
        out.data_ptr(), *os_, _ptr(lse), _ptr(workspace), nbytes, _ptr(err_flag), _stream(stream))
    _check("kvx_paged_attention", st)


def kvx_attention_mass(query, kv_cache, block_table, q_offsets, context_lens, lse, mass,
                       scale: Optional[float] = None, causal: bool = True, window: int = 0,
                       max_query_len: Optional[int] = None, max_context_len: Optional[int] = None,
                       layout: str = "blocks_tokens_kv", err_flag=None, stream=None):
    """Add to mass (float32 [num_reqs][num_kv_heads][width]) the attention weight that the batch's
    queries give to every cached token, summed over the query heads of each KV head; lse is
    kvx_paged_attention's."""
    c = _cache(kv_cache, layout)
    b, heads, qs = _batch(query, c, block_table, q_offsets, context_lens, max_query_len, max_context_len)
    _want_lse(lse, b.num_tokens, heads)
    m = _lists(mass, "mass", b.num_reqs, c.num_kv_heads)
    _on_current_device((query, c.tensor, block_table, q_offsets, context_lens, lse, mass, err_flag))
    st = _F["kvx_attention_mass"](
        c, b, query.data_ptr(), *qs, heads, c.head_dim ** -0.5 if scale is None else float(scale), bool(causal), int(window),
        lse.data_ptr(), mass.data_ptr(), *m, _ptr(err_flag), _stream(stream))
    _check("kvx_attention_mass", st)


def kvx_evict_select(mass, context_lens, budget: int, sink: int, recent: int, keep, new_lens, err_flag=None,
                     stream=None):
    """Per request and head of mass ([num_reqs][heads][width]): the slots that stay, ascending and
    then -1, into keep (int32 [num_reqs][heads][budget]); min(context, budget) into new_lens."""
    import torch

    _want(context_lens, torch.int64, "context_lens")
    _want(keep, torch.int32, "keep")
    _want(new_lens, torch.int64, "new_lens")
    R = context_lens.numel()
    m = _lists(mass, "mass", R, None)
    heads = mass.shape[1]
    if tuple(keep.shape) != (R, heads, int(budget)) or new_lens.numel() != R:
        raise ValueError("kvx: keep must be [num_reqs][heads][budget] and new_lens [num_reqs]")
    _on_current_device((mass, context_lens, keep, new_lens, err_flag))
    st = _F["kvx_evict_select"](mass.data_ptr(), *m, R, heads, context_lens.data_ptr(), int(budget), int(sink), int(recent),
                                keep.data_ptr(), new_lens.data_ptr(), _ptr(err_flag), _stream(stream))
    _check("kvx_evict_select", st)


def kvx_evict_compact(kv_cache, block_table, dst_block_table, keep, mass=None, mass_out=None,
                      layout: str = "blocks_tokens_kv", err_flag=None, stream=None):
    """Move the kept slots' K and V rows (and masses) together, slot keep[r][h][i] to slot i of
    dst_block_table: block_table itself (the same tensor, whole) for a move in place, else a table of
    blocks none of which is a source block. A copy of block_table is not in place: rows that would
    move within it are skipped and raise DEVERR_BLOCK_RANGE."""
    import torch

    c = _cache(kv_cache, layout)
    _want(keep, torch.int32, "keep")
    shape = keep.shape
    if len(shape) != 3:
        raise ValueError("kvx: keep must be [num_reqs][heads][budget]")
    R, heads, budget = shape
    src, dst = _table(block_table, R), _table(dst_block_table, R, "dst_block_table")
    if heads == 0 or c.num_kv_heads % heads:
        raise ValueError("kvx: the KV heads must be a multiple of the heads that chose")
    if (mass is None) != (mass_out is None):
        raise ValueError("kvx: mass and mass_out go together")
    m, mo, m_ptr, mo_ptr = (0, 0, 0), (0, 0, 0), None, None
    if mass is not None:
        m, mo = _lists(mass, "mass", R, heads), _lists(mass_out, "mass_out", R, heads)
        m_ptr, mo_ptr = mass.data_ptr(), mass_out.data_ptr()
    _on_current_device((c.tensor, block_table, dst_block_table, keep, mass, mass_out, err_flag))
    st = _F["kvx_evict_compact"](c, block_table.data_ptr(), *src, dst_block_table.data_ptr(), *dst, R, heads,
                                 keep.data_ptr(), budget, m_ptr, *m, mo_ptr, *mo, _ptr(err_flag), _stream(stream))
    _check("kvx_evict_compact", st)
