"""The 4-bit cache format in 64 bits on the CPU, and inputs and results of the calls of include/kvx_fp4.h
for the GPU tests. Nothing here shares code with the kernels."""
from __future__ import annotations

import math

import numpy as np
import torch

import attention_util as A
from gpu_util import DEV, kvx

LAYOUTS4 = ("blocks_heads_kv", "blocks_kv_heads", "kv_blocks_heads")
MOST = {torch.bfloat16: 125, torch.float16: 13}
VALUES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)


def plane_bytes(block, dim):
    return -(-block * (dim // 2 + dim // 32) // 16) * 16


def quantise(x, most):
    """(codes uint8 [..., dim], scale bytes uint8 [..., dim/32]) of rows in 64 bits, by search: the smallest
    exponent that keeps the largest magnitude below 7, then the nearest of the eight values, of two as near the even code."""
    x = np.asarray(x, np.float64)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    top = np.abs(g).max(-1)
    bad = ~np.isfinite(top)
    e = np.full(top.shape, most)
    for k in range(most - 1, -128, -1):  # downwards while the next smaller one still does
        e = np.where((e == k + 1) & (top < 7 * 2.0 ** k), k, e)
    with np.errstate(all="ignore"):
        y = np.abs(g / 2.0 ** e[..., None])
        dist = np.abs(y[..., None] - VALUES)
        near = dist == dist.min(-1, keepdims=True)
        even = np.arange(8) % 2 == 0
        codes = np.where((near & even).any(-1), (near & even).argmax(-1), near.argmax(-1))
    codes = codes + 8 * np.signbit(g)
    codes = np.where(bad[..., None], 0, codes).astype(np.uint8)
    return codes.reshape(x.shape), np.where(bad, 255, e + 127).astype(np.uint8)


def values(codes, scales):
    """What they stand for, in 64 bits."""
    c = codes.reshape(*codes.shape[:-1], codes.shape[-1] // 32, 32)
    v = np.where(c >= 8, -1.0, 1.0) * VALUES[c & 7]
    p = np.where(scales == 255, math.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (v * p[..., None]).reshape(codes.shape)


def to_planes(codes, scales):
    """codes [..., block, dim] and scales [..., block, dim/32] as plane bytes (the filling is 0xcd)."""
    block, dim = codes.shape[-2:]
    lead = codes.shape[:-2]
    out = np.full((*lead, plane_bytes(block, dim)), 0xcd, np.uint8)
    n, s = block * dim // 2, block * dim // 32
    out[..., :n] = (codes[..., 0::2] | codes[..., 1::2] << 4).reshape(*lead, n)
    out[..., n:n + s] = scales.reshape(*lead, s)
    return out


def from_planes(planes, block, dim):
    """(codes, scales) of plane bytes."""
    lead = planes.shape[:-1]
    n, s = block * dim // 2, block * dim // 32
    b = planes[..., :n].reshape(*lead, block, dim // 2)
    codes = np.stack([b & 15, b >> 4], -1).reshape(*lead, block, dim)
    return codes, planes[..., n:n + s].reshape(*lead, block, dim // 32)


def as_planes(cache, layout):
    """[blocks][heads][K, V][plane], a view (tensor or array)."""
    t = torch.from_numpy(cache) if isinstance(cache, np.ndarray) else cache
    t = t if layout == LAYOUTS4[0] else t.transpose(1, 2) if layout == LAYOUTS4[1] else t.permute(1, 2, 0, 3)
    return t.numpy() if isinstance(cache, np.ndarray) else t


def shape_of(blocks, heads, plane, layout):
    return {LAYOUTS4[0]: (blocks, heads, 2, plane), LAYOUTS4[1]: (blocks, 2, heads, plane),
            LAYOUTS4[2]: (2, blocks, heads, plane)}[layout]


class Case4(A.Case):
    """A batch over a 4-bit cache on the host; slots that no context covers have NaN scales. `cache` is a uint8
    tensor that to() sends to the device."""

    def __init__(self, seed, lens, heads=4, kv_heads=2, dim=64, block=16, dtype="bf16", layout=LAYOUTS4[0], extra=0, spare=3,
                 q_scale=1.5):
        super().__init__(seed, lens, heads, kv_heads, dim, block, dtype, A.LAYOUTS[0], extra, spare, q_scale)
        rows = self.cache.double().numpy().transpose(0, 3, 2, 1, 4)  # [blocks][heads][K, V][block][dim]
        rng = np.random.default_rng(seed + 1)
        gain = np.where(rng.random(dim) < 0.1, 4.0, 1.0)  # some channels stand out
        codes, scales = quantise(rows * gain, MOST[self.dtype])
        self.layout = layout
        plane = plane_bytes(block, dim)
        cache = np.zeros(shape_of(self.num_blocks, kv_heads, plane, layout), np.uint8)
        as_planes(cache, layout)[:] = to_planes(codes, scales)
        self.cache = torch.from_numpy(cache)

    def planes(self):
        return as_planes(self.cache.numpy(), self.layout)

    def set_scale(self, r, slot, head, w, group, byte, code=None):
        """One group's scale byte of request r's slot, and all its codes."""
        n = self.block * self.dim // 2
        b = self.table[r, slot // self.block]
        if code is not None:
            at = slot % self.block * self.dim // 2 + group * 16
            self.planes()[b, head, w, at:at + 16] = code | code << 4
        self.planes()[b, head, w, n + slot % self.block * (self.dim // 32) + group] = byte

    def rows_of(self, r):
        c = min(max(int(self.context[r]), 0), self.width * self.block)
        j = np.arange(c)
        ids = self.table[r, j // self.block].astype(np.int64)
        ok = (ids >= 0) & (ids < self.num_blocks)
        codes, scales = from_planes(self.planes()[np.where(ok, ids, 0)], self.block, self.dim)  # [slots][heads][K, V][block][..]
        at = np.arange(c)[:, None, None], np.arange(self.kv_heads)[None, :, None], np.arange(2)[None, None, :], (j % self.block)[:, None, None]
        v = values(codes[at], scales[at])  # [slots][heads][K, V][dim]
        kv = torch.from_numpy(np.ascontiguousarray(v.transpose(0, 2, 1, 3)))
        return kv.to(self.dtype).double(), torch.from_numpy(ok)  # values are taken in the 16-bit type


def attention(case: Case4, causal=True, window=0, scale=None):
    """attention_util.attention, and what its bound leaves out where a slot's weight is next to nothing: the hardware's
    exponential has no subnormal results, so a weight below 2^-126 of the largest is lost whole. c slots lose at most
    c 2^-126 max|v|. (Seen at scores 90 apart, exp(-90) = 2^-130: 3.6e-40 came out as 0.)"""
    out, lse, tol, tol_lse = A.attention(case, causal, window, scale)
    group = case.heads // case.kv_heads
    for r, (n, _) in enumerate(case.lens):
        v = case.rows_of(r)[0][:, 1].nan_to_num(0, 0, 0).abs()
        if n and v.shape[0]:
            at = slice(int(case.offsets[r]), int(case.offsets[r]) + n)
            tol[at] += v.shape[0] * 2.0 ** -126 * v.amax((0, 2)).repeat_interleave(group)[None, :, None]
    return out, lse, tol, tol_lse


def attend(case: Case4, dev, causal=True, window=0, scale=None, split=True, out=None, hints=True, stream=None, workspace=None):
    """The call on the device tensors of case.to(): (out, lse, error bits)."""
    K = kvx()
    q, cache, table, offsets, context = dev
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device=q.device) if out is None else out
    lse = torch.full(q.shape[:2], 7.0, device=q.device)
    err = torch.zeros(1, dtype=torch.int32, device=q.device)
    n, c = max([n for n, _ in case.lens] + [0]), max(list(case.context) + [0])
    if split:
        c = max(int(c), 2000)  # a hint may be high: short contexts are shared out as well
    ws = workspace
    if ws is None and split:
        ws = K.new_attention_workspace_fp4(q, cache, len(case.lens), n, max(int(c), 0), layout=case.layout)
    K.kvx_paged_attention_fp4(q, cache, table, offsets, context, out, lse, scale=scale, causal=causal, window=window,
                              workspace=ws, layout=case.layout, err_flag=err, max_query_len=n if hints else None,
                              max_context_len=max(int(c), 0) if hints else None, stream=stream)
    torch.cuda.synchronize()
    return out, lse, int(err.item())
