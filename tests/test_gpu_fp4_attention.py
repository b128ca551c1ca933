"""kvx_paged_attention_fp4 against float64 results over what the cache's bytes stand for: types, head layouts, lengths, masks,
blocks, scales at their ends, bad tables and offsets, and workspaces."""
import math

import numpy as np
import pytest
import torch

import attention_util as A
import fp4_util as F
from gpu_util import DEV, kvx, log

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    log(f"start {request.node.name}")
    yield
    torch.cuda.synchronize()


def run(case, causal=True, window=0, scale=None, split=True, hints=True, err=0):
    out, lse, got_err = F.attend(case, case.to(), causal, window, scale, split=split, hints=hints)
    assert got_err == err
    want, want_lse, tol, tol_lse = F.attention(case, causal, window, scale)
    nobody = want.isnan().all(-1) & want_lse.isnan()
    n = int(case.offsets[-1])
    nobody[:n] = False
    A.check("out", out.cpu()[:n], want[:n], tol[:n])
    A.check("lse", lse.cpu()[:n], want_lse[:n], tol_lse[:n])
    assert bool((out.cpu()[n:] == 7).all()) and bool((lse.cpu()[n:] == 7).all()), "rows of nobody were written"
    return out, lse


DECODE = [(1, 1), (1, 2), (1, 17), (1, 700), (1, 64), (1, 129)]
MIXED = [(1, 40), (5, 5), (0, 9), (3, 300), (70, 200), (1, 1), (130, 513), (2, 2)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 256])
def test_decode_dims(dim, dtype):
    run(F.Case4(1, DECODE, dim=dim, dtype=dtype))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 192, 256])
def test_mixed_dims(dim, dtype):
    run(F.Case4(2, MIXED, dim=dim, dtype=dtype, extra=3))


@pytest.mark.parametrize("heads,kv", [(1, 1), (8, 8), (8, 1), (7, 1), (15, 3), (16, 1), (17, 1), (24, 1), (40, 2), (64, 2)])
@pytest.mark.parametrize("lens", [[(1, 90), (1, 260)], [(2, 31), (1, 150)], [(9, 200), (40, 40)]])
def test_head_groups(heads, kv, lens):
    run(F.Case4(3, lens, heads=heads, kv_heads=kv, dim=64))


@pytest.mark.parametrize("block", [1, 3, 8, 16, 24, 64])
@pytest.mark.parametrize("layout", F.LAYOUTS4)
def test_blocks_and_layouts(block, layout):
    run(F.Case4(4, [(1, 33), (20, 150), (1, 500)], block=block, layout=layout, dim=96))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 15, 64, 200])
@pytest.mark.parametrize("lens", [DECODE, MIXED])
def test_masks(causal, window, lens):
    run(F.Case4(5, lens, dtype="fp16"), causal=causal, window=window)


def test_more_tokens_than_slots():
    """Rows whose mask leaves nothing: out 0, lse -inf."""
    case = F.Case4(6, [(9, 4), (3, 0), (200, 150), (1, 0)])
    out, lse = run(case)
    assert bool((out[:5] == 0).all()) and bool((lse[:5] == -math.inf).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("lens", [[(1, 3000), (1, 5)], [(1, 9000)], [(1, 1500)] * 5 + [(1, 60)], [(4, 2500), (3, 100)], [(100, 2600), (60, 60)]])
@pytest.mark.parametrize("split", [True, False])
def test_split_contexts(lens, split, dtype):
    run(F.Case4(7, lens, heads=8, kv_heads=1, dim=128, dtype=dtype), split=split)


@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("lens", [[(9, 100), (16, 2700), (1, 5), (0, 3), (12, 12)], [(11, 40), (13, 1300)]])
def test_several_tiles_of_few_rows(lens, split):
    """33 to 64 rows a request: two tiles of 32."""
    run(F.Case4(21, lens, heads=8, kv_heads=2, dim=128), split=split)
    run(F.Case4(21, lens, heads=8, kv_heads=2, dim=64, dtype="fp16"), split=split, window=30)


@pytest.mark.parametrize("window", [900, 1000, 1500, 2300])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens", [[(1, 2700), (3, 1500), (2, 950)], [(1, 2700), (70, 2000), (20, 20), (2, 950)]])
def test_windows_in_split_contexts(lens, causal, window):
    run(F.Case4(25, lens, heads=4, kv_heads=2, dim=64), causal=causal, window=window)


@pytest.mark.parametrize("split", [True, False])
def test_three_tiles_of_few_rows(split):
    run(F.Case4(22, [(24, 500), (3, 1900), (17, 30)], heads=4, kv_heads=1, dim=256), split=split)


@pytest.mark.parametrize("window,causal", [(0, True), (0, False), (200, True)])
def test_shares_of_tiles_that_fill_the_gpu(window, causal):
    """640 and 768 tiles of 128 rows, shared out to 512 workgroups (with the window: not)."""
    run(F.Case4(23, [(129, 700), (129, 130), (140, 600), (5, 700), (0, 9), (129, 333)], heads=64, kv_heads=64, dim=64, dtype="fp16"),
        window=window, causal=causal)
    if not window:
        run(F.Case4(24, [(1100, 5000)], heads=64, kv_heads=64, dim=32), causal=causal, scale=0.3)


def test_many_requests():
    rng = np.random.default_rng(8)
    lens = [(int(rng.integers(0, 4)), int(rng.integers(0, 90))) for _ in range(150)]
    run(F.Case4(8, lens, heads=4, kv_heads=2, dim=32))


@pytest.mark.parametrize("lens", [DECODE, MIXED])
def test_wrong_hints_change_nothing(lens):
    case = F.Case4(9, lens)
    run(case, hints=False)
    K, dev = kvx(), case.to()
    want, want_lse, tol, tol_lse = F.attention(case)
    for n, c in ((1, 1), (0, 0), (1, 1 << 40), (1 << 40, 16)):
        q, cache, table, offsets, context = dev
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device=DEV)
        ws = K.new_attention_workspace_fp4(q, cache, len(lens), n, c)
        K.kvx_paged_attention_fp4(q, cache, table, offsets, context, out, lse, max_query_len=n, max_context_len=c, workspace=ws)
        torch.cuda.synchronize()
        A.check("out", out, want, tol)
        A.check("lse", lse, want_lse, tol_lse)


@pytest.mark.parametrize("lens", [[(1, 2000), (1, 900)], [(64, 1700)]])
def test_small_workspaces_and_repeats(lens):
    """A workspace of any size, down to none; the same call gives the same bits."""
    case = F.Case4(10, lens, heads=8, kv_heads=1)
    K, dev = kvx(), case.to()
    want, want_lse, tol, tol_lse = F.attention(case)
    full = K.new_attention_workspace_fp4(dev[0], dev[1], len(lens), lens[0][0], lens[0][1])
    for part in (0, 1, 3, 7, 9, 10):
        n = full.numel() * part // 10 // 16 * 16
        guard = torch.full((n + 64,), 0x5a, dtype=torch.uint8, device=DEV)
        a, l, _ = F.attend(case, dev, workspace=guard[:n])
        assert bool((guard[n:] == 0x5a).all()), "written behind the workspace"
        A.check("out", a, want, tol)
        A.check("lse", l, want_lse, tol_lse)
        b, m, _ = F.attend(case, dev, workspace=guard[:n])
        assert torch.equal(a, b) and torch.equal(l, m)


def test_strided_rows_no_lse_and_struct():
    K, case = kvx(), F.Case4(11, [(3, 50), (1, 80)], heads=6, kv_heads=2, dim=64)
    q, cache, table, offsets, context = case.to()
    fused = torch.zeros(case.T, 10, 64, dtype=q.dtype, device=DEV)
    fused[:, 2:8] = q
    out = torch.full((case.T, 7, 96), 7.0, dtype=q.dtype, device=DEV)
    wide = torch.zeros(2, table.shape[1] + 3, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    held = torch.zeros(cache.shape[0], 5, 2, cache.shape[3], dtype=torch.uint8, device=DEV)
    held[:, 1:3] = cache
    K.kvx_paged_attention_fp4(fused[:, 2:8], K.fp4_cache(held[:, 1:3], 64, torch.bfloat16), wide[:, :table.shape[1]], offsets, context,
                              out[:, :6, 16:80])
    torch.cuda.synchronize()
    want, _, tol, _ = F.attention(case)
    A.check("out", out[:, :6, 16:80], want, tol)
    assert bool((out[:, 6] == 7).all()) and bool((out[:, :, :16] == 7).all()) and bool((out[:, :, 80:] == 7).all())


# ----------------------------------------------------------------------------------------
# scales and values at their ends
# ----------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim", [64, 256])
@pytest.mark.parametrize("lens", [[(1, 200), (1, 31)], [(6, 200), (3, 31)], [(150, 200), (33, 40)]])
def test_nan_and_infinite_slots_reach_only_rows_that_see_them(lens, dim, dtype):
    """NaN scales of K and V, and infinite values of V, in slots that some rows do not see. (Values that are finite but near
    the end of 32 bits' range are another matter: 2^8 times as much is summed up before it is divided.)"""
    case = F.Case4(12, lens, heads=4, kv_heads=2, dim=dim, dtype=dtype)
    n = lens[0][0]
    case.set_scale(0, 200 - n, 0, 1, 0, 255)     # the first new token's own V: all new tokens see it
    case.set_scale(0, 199, 0, 0, dim // 32 - 1, 255)  # the last one's K
    case.set_scale(0, 10, 1, 1, 1, 254, 7)          # outside the window of most
    case.set_scale(0, 199, 1, 1, 0, 253, 14)
    case.set_scale(1, 30, 1, 1, dim // 32 - 1, 255)
    for causal, window in ((True, 0), (True, 20), (False, 7)):
        run(case, causal=causal, window=window)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim", [32, 96, 160, 224])
@pytest.mark.parametrize("lens", [[(1, 200)], [(6, 200)], [(150, 200)]])
def test_infinite_keys_on_the_far_side(lens, dim, dtype):
    """A key that reads back infinite, with a score of minus infinity: its slot weighs nothing, as with one whose score is
    merely far below the others', and heads narrower than the kernels' widths see no infinity times zero."""
    case = F.Case4(13, lens, heads=4, kv_heads=2, dim=dim, dtype=dtype)
    case.q[:, :, :32] = -case.q[:, :, :32].abs() - 0.25
    case.q[:, :, -32:] = -case.q[:, :, -32:].abs() - 0.25
    outs = []
    for byte in (254 if dtype == "bf16" else 150, 138):  # 6 * 2^127 and 6 * 2^23 are infinite in the types, 6 * 2^11 is not
        for head, group in ((0, 0), (1, dim // 32 - 1)):
            case.set_scale(0, 10, head, 0, group, byte, 7)
        outs.append(F.attend(case, case.to()))
    run(case)
    for inf, low in zip(*outs):
        assert inf == low if isinstance(inf, int) else torch.equal(inf, low)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_small_and_large_scales(dtype):
    """K groups near the ends of the scale's range beside ordinary ones; V as far as the type goes."""
    case = F.Case4(13, [(1, 100), (20, 60)], heads=4, kv_heads=2, dim=64, dtype=dtype)
    for j in range(0, 60, 3):
        case.set_scale(0, j, 0, 0, 0, 0)
        case.set_scale(1, j, 1, 0, 1, 1 + j)
        case.set_scale(0, j, 0, 1, 1, 104)
        case.set_scale(1, j, 0, 1, 0, 138 if dtype == "fp16" else 180)
    run(case)


def test_far_scores():
    """Scores of 2^20 and more, in both types: one slot takes all the weight."""
    for dtype in ("bf16", "fp16"):
        for e in (132, 136, 140):
            case = F.Case4(14, [(1, 300), (3, 40), (40, 150)], heads=4, kv_heads=2, dim=64, dtype=dtype, q_scale=40)
            for r, (_, c) in enumerate(case.lens):
                for j in range(5, c, 31):
                    for h in range(2):
                        for grp in range(2):
                            case.set_scale(r, j, h, 0, grp, e)
            run(case)


def test_attention_sink_fp16():
    """A first slot that outweighs each of many others by 2^18: what they weigh together counts."""
    case = F.Case4(15, [(1, 4000), (2, 2000)], heads=4, kv_heads=1, dim=64, dtype="fp16", q_scale=0.02)
    case.q[:] = 0
    case.q[:, :, 0] = 1.0
    planes = case.planes()
    n = 16 * 32
    for r, (_, c) in enumerate(case.lens):
        for j in range(c):
            b = case.table[r, j // 16]
            planes[b, 0, 0, j % 16 * 32] = 0
        b = case.table[r, 0]
        planes[b, 0, 0, 0] = 0x06  # K[0][0] = 4
        planes[b, 0, 0, n] = 127 + 2
    run(case, scale=math.log(2.0) * 18 / 16)


def test_q_rows_of_all_sizes():
    """Rows of q from subnormal to near the largest number, rows of zeros, and rows with one element far above the others."""
    for dtype in ("bf16", "fp16"):
        case = F.Case4(16, [(24, 60)], heads=2, kv_heads=1, dim=64, dtype=dtype)
        big = 2.0 ** (12 if dtype == "fp16" else 30)
        for i in range(24):
            case.q[i] *= 2.0 ** -i if i < 12 else 1.0
        case.q[12], case.q[13] = 0, -0.0
        case.q[14] *= torch.finfo(case.dtype).smallest_normal
        case.q[15, :, 7] = 3000.0
        case.q[16, :, 8] = -1500.0
        run(case, scale=0.01)
        case.q[20] *= big
        run(case, scale=float(2.0 ** -20))


def test_q_rows_that_are_not_finite():
    case = F.Case4(17, [(4, 60)], heads=2, kv_heads=1, dim=64)
    dev = case.to()
    dev[0][1, 0, 5], dev[0][2, 1, 9] = math.inf, math.nan
    out, lse, _ = F.attend(case, dev)
    want, want_lse, tol, tol_lse = F.attention(case)
    for t, h in ((1, 0), (2, 1)):
        assert bool(out[t, h].isnan().all()) and bool(lse[t, h].isnan())
        want[t, h], want_lse[t, h] = math.nan, math.nan
    A.check("out", out, want, tol)
    A.check("lse", lse, want_lse, tol_lse)


# ----------------------------------------------------------------------------------------
# tables, offsets and contexts that are wrong
# ----------------------------------------------------------------------------------------

@pytest.mark.parametrize("lens", [[(1, 100), (1, 300)], [(20, 100), (50, 300)]])
def test_bad_block_ids(lens):
    K, case = kvx(), F.Case4(18, lens)
    case.table[0, 2], case.table[1, 7], case.table[1, 18] = -5, case.num_blocks, 1 << 30
    run(case, err=K.DEVERR_BLOCK_RANGE)


@pytest.mark.parametrize("lens", [[(1, 100), (1, 30)], [(20, 100), (5, 30)]])
def test_bad_contexts(lens):
    K, case = kvx(), F.Case4(19, lens)
    case.context[0], case.context[1] = 100000, -7
    # the first context is cut at the table's width, whose blocks it all has
    case.lens[0] = (lens[0][0], case.width * case.block)
    rng = np.random.default_rng(1)
    case.table[0] = rng.permutation(case.num_blocks)[:case.width]
    codes, _ = F.from_planes(case.planes(), 16, 64)
    F.as_planes(case.cache.numpy(), case.layout)[:] = F.to_planes(codes, np.full((*codes.shape[:-1], 2), 127, np.uint8))
    run(case, err=K.DEVERR_TABLE_RANGE)


@pytest.mark.parametrize("offsets", [[0, 3, 1, 4], [-5, 2, 900, 4], [0, 0, 0, 1 << 40], [3, 2, 1, 0]])
def test_bad_offsets_stay_inside(offsets):
    """Offsets that are no CSR: reported, and nothing outside the tensors is touched."""
    K, case = kvx(), F.Case4(20, [(1, 700), (2, 30), (1, 500)], heads=8, kv_heads=1)
    q, cache, table, _, context = case.to()
    off = torch.tensor(offsets, dtype=torch.int64, device=DEV)
    for n in (1, 40):
        guard = torch.full((case.T + 2, 8, 64), 7.0, dtype=q.dtype, device=DEV)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        size = K.attention_workspace_fp4_bytes(q, cache, 3, n, 700)
        ws = torch.full((size + 256,), 0x5a, dtype=torch.uint8, device=DEV)
        K.kvx_paged_attention_fp4(q, cache, table, off, context, guard[1:-1], workspace=ws[:size], max_query_len=n, max_context_len=700,
                                  err_flag=err)
        torch.cuda.synchronize()
        assert int(err.item()) & K.DEVERR_OFFSETS
        assert bool((guard[0] == 7).all()) and bool((guard[-1] == 7).all()) and bool((ws[size:] == 0x5a).all())


def test_nothing_to_do():
    K = kvx()
    z = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    cache = K.new_fp4_cache(2, 16, 2, 64, DEV)
    off, ctx = torch.zeros(1, dtype=torch.int64, device=DEV), torch.zeros(0, dtype=torch.int64, device=DEV)
    K.kvx_paged_attention_fp4(z, cache, torch.zeros(0, 1, dtype=torch.int32, device=DEV), off, ctx, z)
    q = torch.ones(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    out, lse = torch.full_like(q, 7), torch.full((2, 4), 7.0, device=DEV)
    # a cache without blocks, and a table without columns: nothing is seen
    for nb, cols, c in ((0, 1, 5), (2, 0, 0)):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        K.kvx_paged_attention_fp4(q, K.new_fp4_cache(nb, 16, 2, 64, DEV), torch.zeros(1, cols, dtype=torch.int32, device=DEV),
                                  torch.tensor([0, 2], device=DEV), torch.tensor([c], device=DEV), out, lse, err_flag=err)
        torch.cuda.synchronize()
        assert bool((out == 0).all()) and bool((lse == -math.inf).all()) and int(err.item()) == 0
