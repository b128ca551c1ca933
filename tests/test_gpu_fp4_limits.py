"""The calls of include/kvx_fp4.h at the ends of what they count and hold: scores far from zero, caches past 4 GiB, offsets with more
tiles than 32 bits hold, more layers than a grid has rows."""
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


@pytest.mark.parametrize("split", [False, True], ids=["whole", "shared"])
@pytest.mark.parametrize("n", [1, 8, 70], ids=["decode", "drafts", "chunk"])
@pytest.mark.parametrize("dtype,q_scale,up", [("fp16", 3e3, 6), ("fp16", 8e3, 11), ("bf16", 4e3, 10), ("bf16", 1e5, 14), ("bf16", 1e7, 20)])
def test_scores_far_from_zero(dtype, q_scale, up, n, split):
    """K times 2^up: scores of millions to 10^12, where 32 bits hold a score in steps of 1 to 65536 and the softmax is the slot
    with the largest one."""
    case = F.Case4(80, [(n, n + 900), (n, 2000)], heads=4, kv_heads=1, dim=64, dtype=dtype, q_scale=q_scale)
    s = 16 * 32
    scales = case.planes()[:, :, 0, s:s + 32]
    scales[:] = np.where(scales < 250, scales + up, scales)
    out, lse, bits = F.attend(case, case.to(), split=split)
    assert bits == 0
    h, sure = A.half_step(case.dtype), 0
    for r, (tokens, c) in enumerate(case.lens):
        kv, _ = case.rows_of(r)
        at = slice(int(case.offsets[r]), int(case.offsets[r]) + tokens)
        for head in range(case.heads):
            q, k, v = case.q[at, head].double(), kv[:, 0, 0], kv[:, 1, 0]
            x = (q @ k.t() * case.scale).masked_fill(~case.seen(r, True, 0), -torch.inf)
            best, j = x.topk(2, dim=1)
            # a score is off by (dim + 2) 2^-24 of the sum of its products' sizes, scaling and base 2 add 2^-22
            dx = ((case.dim + 2) * 2.0 ** -24 + 2.0 ** -22) * (q.abs() @ k.abs().t() * case.scale).amax(1)
            # rows whose second best is behind by more than both errors and the 40 that are nothing beside a weight of 1
            clear = best[:, 0] - best[:, 1] > 2 * dx + 40
            sure += int(clear.sum())
            got, want = out[at, head].double().cpu(), v[j[:, 0]]
            assert bool(torch.isfinite(out[at, head]).all()) and bool(torch.isfinite(lse[at, head]).all())
            # one rounding of the weight, one of the result, and sums in 32 bits
            tol = 2 * h * (1 + h) * want.abs() + c * 2.0 ** -24 * want.abs() + torch.finfo(case.dtype).smallest_normal * h
            assert bool(((got - want).abs() <= tol)[clear].all()), (r, head, float((got - want).abs()[clear].max()))
            off = (lse[at, head].double().cpu() - best[:, 0]).abs()
            # where others weigh too, the sum of all of them is at most the number of slots
            assert bool((off <= dx + best[:, 0].abs() * 2.0 ** -22 + 8).all())
    assert sure > 0.8 * case.T * case.heads


@pytest.mark.parametrize("layout", [F.LAYOUTS4[0], F.LAYOUTS4[2]])
def test_caches_past_4_gib(layout):
    """Rows appended to, attended in and read back from the last blocks of a cache of 5 GiB, and what lies 2^32 bytes before them is
    as it was."""
    K = kvx()
    heads, dim, block, T = 2, 128, 16, 37
    plane = F.plane_bytes(block, dim)
    nb = (5 << 30) // (2 * heads * plane)
    cache = K.new_fp4_cache(nb, block, heads, dim, DEV, layout)
    q, k, v, pos, freq, axis = inputs(1, T, 4, heads, dim, 1, dim, "bf16")
    ids = np.array([nb - 1, nb - 7, nb - 2], np.int32)
    slots = torch.from_numpy(ids[np.arange(T) // block].astype(np.int64) * block + np.arange(T) % block).to(DEV)
    qr = torch.empty_like(q, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    K.kvx_rope_and_cache_fp4(q.to(DEV), k.to(DEV), v.to(DEV), pos.to(DEV), freq.to(DEV), axis, slots, cache, qr, layout=layout, err_flag=err)
    torch.cuda.synchronize()
    kv64 = torch.stack([rotated(k, pos, freq, axis, False)[0], v.double()], 2).numpy()
    codes, scales = F.quantise(kv64, 125)
    planes = F.as_planes(cache, layout)
    got_codes, got_scales = F.from_planes(planes[torch.from_numpy(ids.astype(np.int64)).to(DEV)].cpu().numpy(), block, dim)
    for t in range(T):
        assert np.array_equal(got_codes[t // block, :, :, t % block], codes[t]) and np.array_equal(got_scales[t // block, :, :, t % block], scales[t])
    assert int((cache.view(-1)[:1 << 30] != 0).sum()) == 0 and int(err.item()) == 0
    case = F.Case4(1, [(T, T)], 4, heads, dim, block)
    held = torch.from_numpy(F.values(codes, scales).transpose(0, 2, 1, 3).copy())
    case.rows_of = lambda r: (held, torch.ones(T, dtype=torch.bool))
    case.q = qr.cpu()
    want, want_lse, tol, tol_lse = F.attention(case)
    table = torch.from_numpy(ids[None]).to(DEV)
    for a, b in ((0, T), (T - 1, T)):  # tiles of many rows, and of few
        out, lse = torch.empty_like(qr[a:b]), torch.empty(b - a, 4, device=DEV)
        K.kvx_paged_attention_fp4(qr[a:b], cache, table, torch.tensor([0, b - a], device=DEV), torch.tensor([T], device=DEV), out, lse,
                                  layout=layout, max_query_len=b - a, max_context_len=T, err_flag=err)
        torch.cuda.synchronize()
        A.check("out", out, want[a:b], tol[a:b])
        A.check("lse", lse, want_lse[a:b], tol_lse[a:b])
    # the whole cache as a buffer of blocks, of which the list takes three: those of layer 0 are its first ones, so the list counts from there
    layer = torch.zeros(4, block, 2, heads, dim, dtype=torch.bfloat16, device=DEV)
    runs = torch.tensor([[nb - 7, 1, nb - 7, 1]], dtype=torch.int64, device=DEV).repeat(nb, 1)
    K.kvx_unpack_fp4(cache, K.layer_base_table([layer]), layer, runs, torch.ones(1, dtype=torch.int64, device=DEV), nb, buffer_layout=layout,
                     err_flag=err)
    torch.cuda.synchronize()
    assert torch.equal(layer[1].cpu(), held[16:32].to(torch.bfloat16)) and not bool(layer[[0, 2, 3]].any()) and int(err.item()) == 0


def test_bad_offsets_with_more_tiles_than_32_bits():
    """Offsets that give the same 66000 tokens to 32768 requests: 4.3e9 tiles, past 2^32. Nothing is written outside the tensors or
    the workspace, and the bit is raised."""
    K = kvx()
    T, R, heads, guard = 66000, 65535, 32, 1 << 16
    q = torch.zeros(T, heads, 32, dtype=torch.bfloat16, device=DEV)
    cache = K.new_fp4_cache(4, 16, 1, 32, DEV)
    table = torch.zeros(R, 1, dtype=torch.int32, device=DEV)
    off = torch.zeros(R + 1, dtype=torch.int64, device=DEV)
    off[1::2] = T
    ctx = torch.full((R,), 16, dtype=torch.int64, device=DEV)
    out = torch.full((T + 2, heads, 32), 7.0, dtype=torch.bfloat16, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    n = K.attention_workspace_fp4_bytes(q, cache, R, 0, 1 << 20)
    assert n > 0  # the work is shared out, with parts in the workspace
    ws = torch.full((n + 2 * guard,), 0xA5, dtype=torch.uint8, device=DEV)
    K.kvx_paged_attention_fp4(q, cache, table, off, ctx, out[1:T + 1], workspace=ws[guard:guard + n], max_query_len=0,
                              max_context_len=1 << 20, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == K.DEVERR_OFFSETS
    assert bool((ws[:guard] == 0xA5).all()) and bool((ws[guard + n:] == 0xA5).all()), "written outside the workspace"
    assert bool((out[0] == 7).all()) and bool((out[T + 1] == 7).all())


def test_more_layers_than_a_grid_has_rows():
    K = kvx()
    L = 70000
    g = torch.Generator().manual_seed(1)
    layers = [torch.randn((3, 1, 2, 1, 32), generator=g).to(torch.bfloat16).to(DEV) for _ in range(2)]
    bases = K.layer_base_table(layers).repeat(L // 2)
    runs, count = K.new_xfer_list(1, DEV)
    K.kvx_build_xfer_list(torch.tensor([2], dtype=torch.int32, device=DEV), None, torch.tensor([0, 1], device=DEV), K.MODE_PACK, runs, count)
    buf = K.new_fp4_cache(L, 1, 1, 32, DEV)
    K.kvx_pack_fp4(bases, layers[0], runs, count, 1, buf)
    torch.cuda.synchronize()
    for i, layer in enumerate(layers):
        codes, scales = F.quantise(layer[2:].double().cpu().numpy().transpose(0, 3, 2, 1, 4), 125)
        want = torch.from_numpy(F.to_planes(codes, scales)[..., :17])
        got = buf[i::2, :, :, :17].cpu()
        assert torch.equal(got, want.expand_as(got))
