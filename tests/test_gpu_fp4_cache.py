"""kvx_rope_and_cache_fp4, kvx_pack_fp4 and kvx_unpack_fp4 against the format in 64 bits: bytes have to be equal."""
import math

import numpy as np
import pytest
import torch

import attention_util as A
import fp4_util as F
from gpu_util import DEV, kvx, log
from test_gpu_rope import inputs, rotated

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    log(f"start {request.node.name}")
    yield
    torch.cuda.synchronize()


# ----------------------------------------------------------------------------------------
# the write of rotated new rows
# ----------------------------------------------------------------------------------------

def run_append(seed=1, T=37, heads=4, kv=2, dim=64, axes=1, rot=None, dtype="bf16", layout=F.LAYOUTS4[0], block=16,
               interleaved=False, far=None, held=True, edit=None):
    """Rows and their 4-bit form: a key is turned in 64 bits and rounded once, so its bytes are those of the 64-bit
    result (the two differ by 2^-50, and no element of these inputs is that near a border)."""
    K = kvx()
    rot = dim if rot is None else rot
    q, k, v, pos, freq, axis = inputs(seed, T, heads, kv, dim, axes, rot, dtype, far)
    if edit:
        edit(k, v)
    nb = -(-T // block) + 3
    slots = torch.from_numpy(np.random.default_rng(seed).permutation(nb * block)[:T].astype(np.int64))
    slots[1::5] = -1  # padding
    bad = 0
    if T > 6:
        slots[6], bad = nb * block + 2, K.DEVERR_SLOT_RANGE
    plane = F.plane_bytes(block, dim)
    cache = np.full(F.shape_of(nb, kv, plane, layout), 0xab, np.uint8)
    dev = torch.from_numpy(cache.copy()).to(DEV)
    out = torch.full((T + 2, heads, dim), 7.0, dtype=q.dtype, device=DEV)
    ko, vo = (torch.full((T + 2, kv, dim), 7.0, dtype=q.dtype, device=DEV) for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    more = (ko[1:T + 1], vo[1:T + 1]) if held else ()
    K.kvx_rope_and_cache_fp4(q.to(DEV), k.to(DEV), v.to(DEV), pos.to(DEV), freq.to(DEV), axis, slots.to(DEV), dev, out[1:T + 1],
                             *more, layout=layout, interleaved=interleaved, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == bad
    want, tol = rotated(q, pos, freq, axis, interleaved)
    A.check("query", out[1:T + 1], want, tol)
    most = F.MOST[q.dtype]
    kv64 = torch.stack([rotated(k, pos, freq, axis, interleaved)[0], v.double()], 2).numpy()  # [T][heads][K, V][dim]
    codes, scales = F.quantise(kv64, most)
    ok = ((slots >= 0) & (slots < nb * block)).numpy()
    planes = F.as_planes(cache, layout)
    n = block * dim // 2
    rows, ids = (slots.numpy() % block)[ok], (slots.numpy() // block)[ok]
    b = codes[ok][..., 0::2] | codes[ok][..., 1::2] << 4
    for i in range(len(ids)):
        planes[ids[i], :, :, rows[i] * dim // 2:(rows[i] + 1) * dim // 2] = b[i]
        planes[ids[i], :, :, n + rows[i] * dim // 32:n + (rows[i] + 1) * dim // 32] = scales[ok][i]
    got = dev.cpu().numpy()
    assert np.array_equal(got, cache), f"{int((got != cache).sum())} of {cache.size} bytes differ"
    if held:
        v64 = torch.from_numpy(F.values(codes, scales)).to(q.dtype)
        for t, w in ((ko, 0), (vo, 1)):
            x = t[1:T + 1].cpu()
            assert torch.equal(x.isnan(), v64[:, :, w].isnan()) and torch.equal(x.nan_to_num(0), v64[:, :, w].nan_to_num(0))
    for t in (out, ko, vo):
        assert bool((t[0] == 7).all()) and bool((t[T + 1] == 7).all())


@pytest.mark.parametrize("T", [1, 2, 37, 300])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append_lengths(T, dtype):
    run_append(T=T, dtype=dtype, dim=128, heads=8, kv=1)


@pytest.mark.parametrize("axes", [1, 3, 4])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_axes_and_pairings(axes, interleaved):
    run_append(seed=2, axes=axes, interleaved=interleaved, dim=128, held=axes != 3)


@pytest.mark.parametrize("dim,rot", [(32, 32), (32, 16), (64, 16), (96, 80), (96, 96), (128, 64), (160, 48), (256, 256), (256, 112)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_dims_and_partial_rotation(dim, rot, interleaved):
    run_append(seed=3, dim=dim, rot=rot, interleaved=interleaved, axes=2, heads=3, kv=3)


@pytest.mark.parametrize("layout", F.LAYOUTS4)
@pytest.mark.parametrize("block", [1, 3, 16, 24, 64])
def test_append_layouts(layout, block):
    run_append(seed=4, layout=layout, block=block, heads=7, kv=1 if block == 24 else 5, dim=96)


@pytest.mark.parametrize("far", [1 << 20, (1 << 31) - 1])
def test_append_far_positions(far):
    run_append(seed=5, T=60, dim=128, far=far, dtype="fp16", axes=3)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append_extreme_rows(dtype):
    """Zeros, the largest and smallest numbers, infinities and NaN in V, and groups of one magnitude."""
    def edit(k, v):
        v[0], v[2] = 0, -0.0
        v[3] = torch.finfo(v.dtype).max
        v[4] = torch.finfo(v.dtype).smallest_normal * 2.0 ** -4  # subnormal
        v[5, :, 3] = math.nan
        v[7, :, 40] = -math.inf
        v[8] = 7.0
        v[9] = 0.875
        v[10, :, ::2] = -1.75
        k[12] = 0
        k[13, :, 5] = math.nan
        k[14] *= 2.0 ** -10
    run_append(seed=6, T=24, dim=64, heads=2, kv=2, dtype=dtype, edit=edit)


def test_append_keys_alone_in_place_and_strided():
    """query_out = query; no query at all; Q, K and V as slices of one fused projection."""
    K = kvx()
    T, H, Hk, D = 19, 6, 2, 64
    q, k, v, pos, freq, axis = inputs(6, T, H, Hk, D, 1, D, "bf16")
    fused = torch.cat([q, k, v], 1).to(DEV)
    fq, fk, fv = fused[:, :H], fused[:, H:H + Hk], fused[:, H + Hk:]
    slots = torch.arange(T, device=DEV)
    a, b = (K.new_fp4_cache(2, 16, Hk, D, DEV) for _ in range(2))
    K.kvx_rope_and_cache_fp4(None, fk, fv, pos.to(DEV), freq.to(DEV), axis, slots, a, None)
    torch.cuda.synchronize()
    assert torch.equal(fused.cpu(), torch.cat([q, k, v], 1))
    K.kvx_rope_and_cache_fp4(fq, fk, fv, pos.to(DEV), freq.to(DEV), axis, slots, K.fp4_cache(b, D, torch.bfloat16), fq)
    torch.cuda.synchronize()
    want, tol = rotated(q, pos, freq, axis, False)
    A.check("query", fq, want, tol)
    assert torch.equal(a, b) and bool(a.any())


def test_append_no_tokens_and_no_blocks():
    K = kvx()
    z = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    cache = torch.ones_like(K.new_fp4_cache(2, 16, 2, 64, DEV))
    none = torch.zeros(1, 0, dtype=torch.int64, device=DEV)
    K.kvx_rope_and_cache_fp4(z, z, z, none, torch.ones(32, device=DEV), [0] * 32, none[0], cache, z)
    torch.cuda.synchronize()
    assert bool((cache == 1).all())
    one = torch.ones(1, 2, 64, dtype=torch.bfloat16, device=DEV)
    out, err = torch.zeros_like(one), torch.zeros(1, dtype=torch.int32, device=DEV)
    K.kvx_rope_and_cache_fp4(one, one.clone(), one.clone(), torch.zeros(1, 1, dtype=torch.int64, device=DEV), torch.ones(32, device=DEV),
                             [0] * 32, torch.zeros(1, dtype=torch.int64, device=DEV), K.new_fp4_cache(0, 16, 2, 64, DEV), out,
                             err_flag=err)
    torch.cuda.synchronize()
    assert bool((out == 1).all()) and int(err.item()) == K.DEVERR_SLOT_RANGE


# ----------------------------------------------------------------------------------------
# transfer
# ----------------------------------------------------------------------------------------

def run_transfer(seed=1, layers=2, counts=(2, 3, 1), heads=2, dim=64, block=16, dtype="bf16", layout=A.LAYOUTS[0],
                 buffer_layout=F.LAYOUTS4[0], bad=False, edit=None, mode="two"):
    """pack into 4-bit blocks, byte for byte; then unpack into other blocks, value for value; what is not listed stays."""
    K = kvx()
    dt = A.DT[dtype]
    g, rng = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
    N, nb = sum(counts), sum(counts) + 4
    shape = {A.LAYOUTS[0]: (nb, block, 2, heads, dim), A.LAYOUTS[1]: (nb, 2, block, heads, dim), A.LAYOUTS[2]: (2, nb, block, heads, dim)}[layout]
    src = [(torch.randn(shape, generator=g) * 2.0 ** float(rng.integers(-3, 4))).to(dt) for _ in range(layers)]
    if edit:
        edit(src)
    src_ids, dst_ids = (rng.permutation(nb)[:N].astype(np.int32) for _ in range(2))
    src_ids[:2] = np.sort(src_ids[:2])
    if bad and N > 3:
        src_ids[1], dst_ids[3] = nb + 5, -2
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    offsets = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)).to(DEV)
    dsrc, ddst = [t.to(DEV) for t in src], [torch.full(shape, 7.0, dtype=dt, device=DEV) for _ in range(layers)]
    sid, did = torch.from_numpy(src_ids).to(DEV), torch.from_numpy(dst_ids).to(DEV)
    ps, cs = K.new_xfer_list(N, DEV)
    pd, cd = K.new_xfer_list(N, DEV)
    if mode == "direct":
        K.kvx_build_xfer_list(sid, did, offsets, K.MODE_DIRECT, ps, cs)
        pd, cd = ps, cs
    else:
        K.kvx_build_xfer_list(sid, None, offsets, K.MODE_PACK, ps, cs)
        K.kvx_build_xfer_list(None, did, offsets, K.MODE_UNPACK, pd, cd)
    buf = torch.full(F.shape_of(layers * N + 1, heads, F.plane_bytes(block, dim), buffer_layout), 0xcd, dtype=torch.uint8, device=DEV)
    K.kvx_pack_fp4(K.layer_base_table(dsrc), dsrc[0], ps, cs, N, buf, layout=layout, buffer_layout=buffer_layout, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == (K.DEVERR_BLOCK_RANGE if bad else 0)
    planes = F.as_planes(buf.cpu().numpy(), buffer_layout)
    codes, scales = [], []
    for l in range(layers):
        rows = A.as_tokens(src[l], layout).double().numpy().transpose(0, 3, 2, 1, 4)  # [blocks][heads][K, V][tokens][dim]
        ok = (src_ids >= 0) & (src_ids < nb)
        c, s = F.quantise(rows[np.where(ok, src_ids, 0)], F.MOST[dt])
        want = np.where(ok[:, None, None, None], F.to_planes(c, s), 0xcd)
        got = planes[l * N:(l + 1) * N]
        assert np.array_equal(got, want), f"layer {l}: {int((got != want).sum())} of {want.size} bytes differ"
        codes.append(c), scales.append(s)
    assert (planes[layers * N] == 0xcd).all()
    if bad:
        err.zero_()
    K.kvx_unpack_fp4(buf, K.layer_base_table(ddst), ddst[0], pd, cd, N, layout=layout, buffer_layout=buffer_layout, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == (K.DEVERR_BLOCK_RANGE if bad else 0)
    for l in range(layers):
        want = torch.full(shape, 7.0, dtype=dt)
        to = A.as_tokens(want, layout)
        for p in range(N):
            if 0 <= dst_ids[p] < nb and 0 <= src_ids[p] < nb:
                v = torch.from_numpy(F.values(codes[l][p], scales[l][p])).to(dt)  # [heads][K, V][tokens][dim]
                to[int(dst_ids[p])] = v.permute(2, 1, 0, 3)
        got = ddst[l].cpu()
        if bad:  # the block that was not packed holds what the buffer held
            skip = int(dst_ids[1])
            A.as_tokens(got, layout)[skip] = A.as_tokens(want, layout)[skip] = 0
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(0), want.nan_to_num(0)), f"layer {l}"


@pytest.mark.parametrize("dim", [32, 64, 96, 128, 192, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_transfer_dims(dim, dtype):
    run_transfer(dim=dim, dtype=dtype)


@pytest.mark.parametrize("layout", A.LAYOUTS)
@pytest.mark.parametrize("buffer_layout", F.LAYOUTS4)
def test_transfer_layouts(layout, buffer_layout):
    run_transfer(seed=2, layout=layout, buffer_layout=buffer_layout, heads=3, dim=96, block=24)


@pytest.mark.parametrize("block", [1, 2, 3, 8, 64, 100])
def test_transfer_blocks(block):
    run_transfer(seed=3, block=block, heads=1, counts=(1, 4))


@pytest.mark.parametrize("layers,counts", [(1, (1,)), (3, (70, 1, 66)), (5, (9, 0, 40)), (48, (2,))])
def test_transfer_runs(layers, counts):
    run_transfer(seed=4, layers=layers, counts=counts, heads=1, block=8, mode="direct")


def test_transfer_runs_that_leave_the_buffer():
    """The parts of runs inside the buffer move, the others raise the error and touch nothing; of more runs than blocks the
    first count."""
    K = kvx()
    N, nb, block, dim = 6, 9, 16, 64
    src = torch.randn(nb, block, 2, 2, dim, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).to(DEV)
    rows = src.cpu().double().numpy().transpose(0, 3, 2, 1, 4)
    planes = F.to_planes(*F.quantise(rows, F.MOST[torch.bfloat16]))
    ids = {"inside": ([(2, 0, 2), (7, 2, 4)], [2, 3, 7, 8, None, None], 1),  # ids 9 and 10 are past the cache
           "behind": ([(2, 0, 2), (0, 2, 2), (4, 4, 5)], [2, 3, 0, 1, 4, 5], 1), "before": ([(3, -1, 3), (0, 2, 4)], [4, 5, 0, 1, 2, 3], 1),
           "far": ([(1, 0, 2), (0, 1 << 40, 4)], [1, 2] + [None] * 4, 1), "exact": ([(1, 0, 2), (3, 2, 4)], [1, 2, 3, 4, 5, 6], 0)}
    for name, (runs, want, bad) in ids.items():
        log(name)
        table = torch.zeros(N, 4, dtype=torch.int64)
        for i, (b, at, n) in enumerate(runs):
            table[i] = torch.tensor([b, b, at, n])  # the request in the last field's upper half is 0
        xfers, count = table.to(DEV), torch.tensor([len(runs)], dtype=torch.int64, device=DEV)
        buf = torch.full(F.shape_of(N + 1, 2, F.plane_bytes(block, dim), F.LAYOUTS4[0]), 0xcd, dtype=torch.uint8, device=DEV)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        K.kvx_pack_fp4(K.layer_base_table([src]), src, xfers, count, N, buf, err_flag=err)
        assert int(err.item()) == (K.DEVERR_BLOCK_RANGE if bad else 0), name
        got = buf.cpu().numpy()
        for p, b in enumerate(want):
            assert np.array_equal(got[p], np.full_like(got[p], 0xcd) if b is None else planes[b]), (name, p)
        assert (got[N] == 0xcd).all()
        dst = torch.full_like(src, 7.0)
        err.zero_()
        K.kvx_unpack_fp4(buf, K.layer_base_table([dst]), dst, xfers, count, N, err_flag=err)
        assert int(err.item()) == (K.DEVERR_BLOCK_RANGE if bad else 0), name
        held = {b for b in want if b is not None}
        for b in range(nb):
            v = torch.from_numpy(F.values(*F.from_planes(planes[b], block, dim))).permute(2, 1, 0, 3).to(src.dtype)
            assert torch.equal(dst[b].cpu(), v if b in held else torch.full_like(v, 7.0)), (name, b)


def test_transfer_bad_ids():
    run_transfer(seed=5, counts=(3, 5), bad=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_transfer_extreme_values(dtype):
    def edit(src):
        x = src[0].view(-1)
        big, small = torch.finfo(x.dtype).max, torch.finfo(x.dtype).smallest_normal
        for i, v in enumerate([big, -big, big / 2, small, small * 2.0 ** -3, 0.0, -0.0, 7.0, 14.0, 1.75, math.inf, math.nan, -math.inf]):
            x[i * 32::1000] = v
        src[0].view(-1, src[0].shape[-1])[5::9] = 0
    run_transfer(seed=6, dtype=dtype, edit=edit, dim=128)


def test_transfer_every_number():
    """Every bf16 and fp16 number beside a 1, a 7 and a 100 that set the scale."""
    K = kvx()
    for dt in (torch.bfloat16, torch.float16):
        for top in (0.0, 1.0, 7.0, 100.0):
            x = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(dt).view(2, 1024, 2, 1, 16)
            rows = torch.zeros(2, 1024, 2, 1, 32, dtype=dt)
            rows[..., :16], rows[..., 16] = x, top
            src = rows.to(DEV)
            ids = torch.arange(2, dtype=torch.int32, device=DEV)
            runs, count = K.new_xfer_list(2, DEV)
            K.kvx_build_xfer_list(ids, None, torch.tensor([0, 2], device=DEV), K.MODE_PACK, runs, count)
            buf = K.new_fp4_cache(2, 1024, 1, 32, DEV)
            K.kvx_pack_fp4(K.layer_base_table([src]), src, runs, count, 2, buf)
            torch.cuda.synchronize()
            want = F.to_planes(*F.quantise(rows.double().numpy().transpose(0, 3, 2, 1, 4), F.MOST[dt]))
            n = 1024 * 17
            assert np.array_equal(buf.cpu().numpy()[..., :n], want[..., :n])


def test_transfer_nothing():
    K = kvx()
    src = torch.ones(2, 16, 2, 1, 64, dtype=torch.bfloat16, device=DEV)
    runs, count = K.new_xfer_list(1, DEV)
    buf = torch.ones_like(K.new_fp4_cache(2, 16, 1, 64, DEV))
    K.kvx_pack_fp4(K.layer_base_table([src]), src, runs, count, 0, buf)
    K.kvx_pack_fp4(K.layer_base_table([src]), src, runs, count, 1, buf)  # a list with no runs
    K.kvx_unpack_fp4(buf, K.layer_base_table([src]), src, runs, count, 1)
    torch.cuda.synchronize()
    assert bool((buf == 1).all()) and bool((src == 1).all())
