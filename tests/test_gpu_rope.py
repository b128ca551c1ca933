"""kvx_rope_and_cache against float64 results: axes, pairings, partial rotations, layouts, padding,
and positions so far that a 32-bit angle would be off by radians."""
import math

import numpy as np
import pytest
import torch

import attention_util as A
from gpu_util import DEV, kvx, log

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    log(f"start {request.node.name}")
    yield
    torch.cuda.synchronize()


def rotated(x, positions, inv_freq, pair_axis, interleaved):
    """[tokens][heads][dim] turned in 64 bits, and the tolerance: the angle's fraction of a turn is
    kept in 32 bits (2^-24 x pi, and as much again in cos and sin), so each product is off by at most
    2^-21 of |x| + |y|; one rounding to the type."""
    half = len(pair_axis)
    angle = positions.double()[torch.tensor(pair_axis)].t() * inv_freq.double()
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    y = x.double().clone()
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    p, q = x[..., a].double(), x[..., b].double()
    y[..., a], y[..., b] = p * cos - q * sin, q * cos + p * sin
    tol = torch.zeros_like(y)
    tiny = torch.finfo(x.dtype).smallest_normal * A.half_step(x.dtype)
    for s in (a, b):
        tol[..., s] = (p.abs() + q.abs()) * 2.0 ** -21 + y[..., s].abs() * A.half_step(x.dtype) * (1 + 2.0 ** -20) + tiny
    return y, tol


def inputs(seed, T, heads, kv, dim, axes, rot, dtype, far=None):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn((T, n, dim), generator=g).to(A.DT[dtype]) for n in (heads, kv, kv))
    top = far or 40000
    pos = torch.randint(0, top, (axes, T), generator=g)
    if far:
        pos[:, ::3] = far - 1 - torch.arange(pos[:, ::3].shape[1])
        pos[:, 1::3] *= -1
    freq = (1e4 ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))).float()
    axis = [int(i) for i in np.random.default_rng(seed).integers(0, axes, rot // 2)]
    return q, k, v, pos, freq, axis


def run(seed=1, T=37, heads=4, kv=2, dim=64, axes=1, rot=None, dtype="bf16", layout=A.LAYOUTS[0], block=16, interleaved=False,
        far=None):
    K = kvx()
    rot = dim if rot is None else rot
    q, k, v, pos, freq, axis = inputs(seed, T, heads, kv, dim, axes, rot, dtype, far)
    nb = -(-T // block) + 3
    slots = torch.from_numpy(np.random.default_rng(seed).permutation(nb * block)[:T].astype(np.int64))
    slots[1::5] = -1  # padding
    bad = 0
    if T > 6:
        slots[6], bad = nb * block + 2, K.DEVERR_SLOT_RANGE
    shape = {A.LAYOUTS[0]: (nb, block, 2, kv, dim), A.LAYOUTS[1]: (nb, 2, block, kv, dim), A.LAYOUTS[2]: (2, nb, block, kv, dim)}[layout]
    cache = torch.full(shape, math.nan, dtype=A.DT[dtype])
    dev = cache.to(DEV)
    out = torch.full((T + 2, heads, dim), 7.0, dtype=q.dtype, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    K.kvx_rope_and_cache(q.to(DEV), k.to(DEV), v.to(DEV), pos.to(DEV), freq.to(DEV), axis, slots.to(DEV), dev, out[1:T + 1],
                         layout=layout, interleaved=interleaved, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == bad
    want, tol = rotated(q, pos, freq, axis, interleaved)
    A.check("query", out[1:T + 1], want, tol)
    if rot < dim:
        assert torch.equal(out[1:T + 1, :, rot:].cpu(), q[..., rot:])
    assert bool((out[0] == 7).all()) and bool((out[T + 1] == 7).all())
    want_k, tol_k = rotated(k, pos, freq, axis, interleaved)
    got = A.as_tokens(dev.cpu(), layout)
    written = torch.zeros(nb, block, dtype=torch.bool)
    ok = (slots >= 0) & (slots < nb * block)
    b, o = slots[ok] // block, slots[ok] % block
    written[b, o] = True
    A.check("K", got[b, o, 0], want_k[ok], tol_k[ok])
    assert torch.equal(got[b, o, 1].view(torch.int16), v[ok].view(torch.int16)), "V rows"
    assert bool(got[~written].isnan().all()), "other slots were written"


@pytest.mark.parametrize("T", [1, 2, 37, 300])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_lengths(T, dtype):
    run(T=T, dtype=dtype, dim=128, heads=8, kv=1)


@pytest.mark.parametrize("axes", [1, 2, 3, 4])
@pytest.mark.parametrize("interleaved", [False, True])
def test_axes_and_pairings(axes, interleaved):
    run(seed=2, axes=axes, interleaved=interleaved, dim=128)


@pytest.mark.parametrize("dim,rot", [(16, 16), (24, 16), (40, 32), (64, 16), (80, 80), (128, 64), (136, 128), (256, 256), (256, 48)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_dims_and_partial_rotation(dim, rot, interleaved):
    run(seed=3, dim=dim, rot=rot, interleaved=interleaved, axes=2, heads=3, kv=3)


@pytest.mark.parametrize("layout", A.LAYOUTS)
@pytest.mark.parametrize("block", [1, 3, 16, 64])
def test_layouts(layout, block):
    run(seed=4, layout=layout, block=block, heads=7, kv=1)


@pytest.mark.parametrize("far", [1 << 20, (1 << 31) - 1])
def test_far_positions(far):
    """Angles of 2^20 and 2^31 radians: pair 0 turns by the position itself."""
    run(seed=5, T=60, dim=128, far=far, dtype="fp16", axes=3)


def test_in_place_keys_alone_and_strided():
    """query_out = query; no query at all; Q, K and V as slices of one fused projection."""
    K = kvx()
    T, H, Hk, D = 19, 6, 2, 64
    q, k, v, pos, freq, axis = inputs(6, T, H, Hk, D, 1, D, "bf16")
    fused = torch.cat([q, k, v], 1).to(DEV)
    fq, fk, fv = fused[:, :H], fused[:, H:H + Hk], fused[:, H + Hk:]
    slots = torch.arange(T, device=DEV)
    a, b = (torch.zeros(2, 16, 2, Hk, D, dtype=q.dtype, device=DEV) for _ in range(2))
    K.kvx_rope_and_cache(None, fk, fv, pos.to(DEV), freq.to(DEV), axis, slots, a, None)
    torch.cuda.synchronize()
    assert torch.equal(fused.cpu(), torch.cat([q, k, v], 1))
    K.kvx_rope_and_cache(fq, fk, fv, pos.to(DEV), freq.to(DEV), axis, slots, b, fq)
    torch.cuda.synchronize()
    want, tol = rotated(q, pos, freq, axis, False)
    A.check("query", fq, want, tol)
    want_k, tol_k = rotated(k, pos, freq, axis, False)
    A.check("K", a.view(32, 2, Hk, D)[:T, 0], want_k, tol_k)
    assert torch.equal(a, b)


def test_agrees_with_the_plain_write_at_position_zero():
    """Angle 0 turns nothing: the same bytes as kvx_reshape_and_cache."""
    K = kvx()
    q, k, v, pos, freq, axis = inputs(7, 33, 4, 2, 64, 1, 64, "bf16")
    slots = torch.randperm(48)[:33].to(DEV)
    a, b = (torch.full((3, 16, 2, 2, 64), 9.0, dtype=k.dtype, device=DEV) for _ in range(2))
    out = torch.empty_like(q, device=DEV)
    K.kvx_rope_and_cache(q.to(DEV), k.to(DEV), v.to(DEV), torch.zeros_like(pos).to(DEV), freq.to(DEV), axis, slots, a, out)
    K.kvx_reshape_and_cache(k.to(DEV), v.to(DEV), slots, b, *K.cache_strides(b))
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(out.cpu(), q)


def test_no_tokens():
    K = kvx()
    z = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    cache = torch.ones(2, 16, 2, 2, 64, dtype=torch.bfloat16, device=DEV)
    K.kvx_rope_and_cache(z, z, z, torch.zeros(1, 0, dtype=torch.int64, device=DEV), torch.ones(32, device=DEV), [0] * 32,
                         torch.zeros(0, dtype=torch.int64, device=DEV), cache, z)
    torch.cuda.synchronize()
    assert bool((cache == 1).all())
