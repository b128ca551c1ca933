"""Inputs and 64-bit results of the calls that compute on a paged cache, for the GPU tests. The
results come from float64 tensors on the CPU, request by request, and share nothing with the
kernels; how far a kernel may be off is derived next to each of them."""
from __future__ import annotations

import math

import numpy as np
import torch

from gpu_util import DEV, kvx

LAYOUTS = ("blocks_tokens_kv", "blocks_kv_tokens", "kv_blocks_tokens")
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def half_step(dtype) -> float:
    """Largest relative error of one rounding to the type."""
    return torch.finfo(dtype).eps / 2


def as_tokens(cache, layout):
    """The cache as [blocks][tokens][K, V][heads][dim], a view."""
    if layout == "blocks_kv_tokens":
        return cache.permute(0, 2, 1, 3, 4)
    if layout == "kv_blocks_tokens":
        return cache.permute(1, 2, 0, 3, 4)
    return cache


class Case:
    """A batch on the host: lens is a list of (new tokens, context) per request. Slots that no
    context covers hold NaN. `extra` query rows behind the last request belong to nobody."""

    def __init__(self, seed, lens, heads=4, kv_heads=2, dim=64, block=16, dtype="bf16", layout=LAYOUTS[0], extra=0,
                 spare=3, q_scale=1.5):
        self.lens, self.heads, self.kv_heads, self.dim, self.block = list(lens), heads, kv_heads, dim, block
        self.dtype, self.layout = DT[dtype], layout
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        counts = [-(-max(c, 0) // block) for _, c in lens]
        nb = sum(counts) + spare
        self.num_blocks, self.width = nb, max(counts + [1])
        ids = rng.permutation(nb).astype(np.int32)
        self.table = np.full((len(lens), self.width), -1, np.int32)
        shape = {LAYOUTS[0]: (nb, block, 2, kv_heads, dim), LAYOUTS[1]: (nb, 2, block, kv_heads, dim),
                 LAYOUTS[2]: (2, nb, block, kv_heads, dim)}[layout]
        self.cache = torch.full(shape, math.nan, dtype=self.dtype)
        rows = as_tokens(self.cache, layout)
        at = 0
        for r, (_, c) in enumerate(lens):
            self.table[r, :counts[r]] = ids[at:at + counts[r]]
            at += counts[r]
            b, o = self.where(r, np.arange(c))
            rows[b, o] = torch.randn((c, 2, kv_heads, dim), generator=g).to(self.dtype)
        self.offsets = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int64)
        self.T = int(self.offsets[-1]) + extra
        self.q = (torch.randn((self.T, heads, dim), generator=g) * q_scale).to(self.dtype)
        self.context = np.array([c for _, c in lens], np.int64)
        self.scale = dim ** -0.5

    def where(self, r, slots):
        slots = np.asarray(slots)
        return torch.from_numpy(self.table[r, slots // self.block].astype(np.int64)), torch.from_numpy(slots % self.block)

    def rows_of(self, r):
        """K and V of request r's context in 64 bits: [context][2][kv_heads][dim], and which slots
        have a block of the cache."""
        c = min(max(int(self.context[r]), 0), self.width * self.block)
        ids = self.table[r, np.arange(c) // self.block].astype(np.int64)
        ok = (ids >= 0) & (ids < self.num_blocks)
        b = torch.from_numpy(np.where(ok, ids, 0))
        kv = as_tokens(self.cache, self.layout)[b, torch.from_numpy(np.arange(c) % self.block)].double()
        return kv, torch.from_numpy(ok)

    def seen(self, r, causal, window):
        n, c = self.lens[r][0], min(max(int(self.context[r]), 0), self.width * self.block)
        i, j = torch.arange(n)[:, None], torch.arange(c)[None, :]
        last = c - n + i if causal else torch.full((n, 1), c - 1)
        s = j <= last
        return s & (j > last - window) if window else s

    def to(self, device=DEV):
        """The device tensors of a call: query, cache, table, offsets, contexts."""
        return (self.q.to(device), self.cache.to(device), torch.from_numpy(self.table).to(device),
                torch.from_numpy(self.offsets).to(device), torch.from_numpy(self.context).to(device))


def attention(case: Case, causal=True, window=0, scale=None):
    """(out, lse, out tolerance, lse tolerance) in 64 bits; rows of nobody are NaN.

    A score is a sum of dim products in 32 bits: off by at most (dim + 2) 2^-24 sum|q k| scale, and
    its scaling to base 2 adds 2^-22 |x|: together dx, of the row's largest. A weight is then off by
    2 dx + 2^-21 (its own score, the total's, exp2 and sums of partial maxima), by one rounding to
    the element type, and the sums over n slots by n 2^-24 of sum w|v|. fp16 weights below 2^-14 of
    the largest lose up to 2^-25 each. The result is rounded once, to the type, whose smallest step
    is also an error near zero."""
    scale = case.scale if scale is None else scale
    group = case.heads // case.kv_heads
    out = torch.full((case.T, case.heads, case.dim), math.nan, dtype=torch.float64)
    lse = torch.full((case.T, case.heads), math.nan, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    h_ = half_step(case.dtype)
    tiny = torch.finfo(case.dtype).smallest_normal * h_
    for r, (n, _) in enumerate(case.lens):
        if n == 0:
            continue
        kv, ok = case.rows_of(r)
        seen = case.seen(r, causal, window) & ok[None, :]
        at = slice(int(case.offsets[r]), int(case.offsets[r]) + n)
        c = kv.shape[0]
        for h in range(case.heads):
            q, k, v = case.q[at, h].double(), kv[:, 0, h // group], kv[:, 1, h // group]
            x = torch.where(seen, q @ k.nan_to_num(0, 0, 0).t() * scale, -math.inf)
            x = torch.where(seen & ~torch.isfinite(k).all(1)[None], (q[:, None, :] * k[None]).sum(-1) * scale, x) \
                if not torch.isfinite(k).all() else x
            some = seen.any(1)
            l = torch.where(some, torch.logsumexp(x, 1) if c else torch.full((n,), -math.inf, dtype=torch.float64),
                            -math.inf)
            w = torch.where(seen, torch.exp(x - torch.where(some, l, 0.0)[:, None]), 0.0)
            if torch.isfinite(v).all():
                o = w @ v
            else:  # a weight of zero outside the mask is no product
                o = torch.where(seen[:, :, None], w[:, :, None] * v[None], 0.0).sum(1)
            out[at, h], lse[at, h] = o, l
            big = (q.abs() @ k.nan_to_num(0, 0, 0).abs().t() * scale).amax(1) if c else torch.zeros(n, dtype=torch.float64)
            dx = (case.dim + 2) * 2.0 ** -24 * big + 2.0 ** -22 * big
            wv = w @ v.nan_to_num(0, 0, 0).abs()
            t = (2 * dx + 2.0 ** -21 + h_ + c * 2.0 ** -24)[:, None] * wv + h_ * o.abs() + tiny
            if case.dtype == torch.float16:
                t = t + c * 2.0 ** -25 * (v.nan_to_num(0, 0, 0).abs().max() if c else 0.0)
            tol[at, h] = t
            tol_lse[at, h] = dx + 2.0 ** -21 + c * 2.0 ** -24 + l.nan_to_num(0, 0, 0).abs() * 2.0 ** -22
    return out, lse, tol, tol_lse


def masses(case: Case, lse, causal=True, window=0, scale=None):
    """(added masses, tolerance, slots some row sees) for given lse [T][heads]: [reqs][kv_heads][width].

    A term exp(x - lse) is off by dx as above and by the roundings of x - lse in base 2, at most
    2^-22 (|x| + |lse|); exp2 by 2^-22; the sum of m terms by m 2^-24, and adding it by half a step."""
    scale = case.scale if scale is None else scale
    group, width = case.heads // case.kv_heads, case.width * case.block
    got = torch.zeros(len(case.lens), case.kv_heads, width, dtype=torch.float64)
    tol, touched = torch.zeros_like(got), torch.zeros(got.shape, dtype=torch.bool)
    for r, (n, _) in enumerate(case.lens):
        kv, ok = case.rows_of(r)
        c = kv.shape[0]
        if n == 0 or c == 0:
            continue
        seen = case.seen(r, causal, window) & ok[None, :]
        at = slice(int(case.offsets[r]), int(case.offsets[r]) + n)
        for h in range(case.heads):
            q, k = case.q[at, h].double(), kv[:, 0, h // group].nan_to_num(0, 0, 0)
            x = q @ k.t() * scale
            l = lse[at, h].double()
            live = seen & (l != -math.inf)[:, None]
            term = torch.where(live, torch.exp(x - torch.where(l == -math.inf, 0.0, l)[:, None]), 0.0)
            big = q.abs() @ k.abs().t() * scale
            rel = (case.dim + 2) * 2.0 ** -24 * big + 2.0 ** -22 * (big + l.nan_to_num(0, 0, 0).abs()[:, None]) + 2.0 ** -21
            got[r, h // group, :c] += term.sum(0)
            tol[r, h // group, :c] += (term * (rel + n * group * 2.0 ** -24)).sum(0)
            touched[r, h // group, :c] |= seen.any(0)
    return got, tol, touched


def check(name, got, want, tol):
    """Every element of got within its tolerance of want, the non-finite ones equal."""
    got, want = got.double().cpu(), want.double()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    fin = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fin), f"{name}: other elements are finite"
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{name}: other elements are NaN"
    inf = ~fin & ~torch.isnan(want)
    assert torch.equal(got[inf], want[inf]), f"{name}: infinities differ"
    off = (got - want).abs()[fin] - tol[fin]
    assert off.numel() == 0 or float(off.max()) <= 0, \
        f"{name}: {int((off > 0).sum())} of {off.numel()} elements off by up to {float((got - want).abs()[fin].max()):.3g}"


def attend(case: Case, dev, causal=True, window=0, scale=None, split=True, out=None, hints=True):
    """The call on the device tensors of case.to(): (out, lse, error bits)."""
    K = kvx()
    q, cache, table, offsets, context = dev
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device=q.device) if out is None else out
    lse = torch.full(q.shape[:2], 7.0, device=q.device)
    err = torch.zeros(1, dtype=torch.int32, device=q.device)
    n, c = max([n for n, _ in case.lens] + [0]), max(list(case.context) + [0])
    ws = K.new_attention_workspace(q, cache, len(case.lens), n, max(int(c), 0), layout=case.layout) if split else None
    K.kvx_paged_attention(q, cache, table, offsets, context, out, lse, scale=scale, causal=causal, window=window,
                          workspace=ws, layout=case.layout, err_flag=err, max_query_len=n if hints else None,
                          max_context_len=max(int(c), 0) if hints else None)
    torch.cuda.synchronize()
    return out, lse, int(err.item())
