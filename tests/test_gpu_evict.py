"""kvx_evict_select and kvx_evict_compact against a plain host selection and row moves, bit for bit;
and the whole chain of a serving loop: rotate and write, attend, accumulate, evict, attend again."""
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


def chosen(mass, n, budget, sink, recent):
    """The kept slots by definition: protected first, then NaN, then by mass, ties to the lowest."""
    if n <= budget:
        return list(range(n))

    def key(j):
        m = float(mass[j])
        if j < sink or j >= n - recent:
            return (0, 0.0, j)
        return (1, 0.0, j) if math.isnan(m) else (2, -m if m != 0 else 0.0, j)
    return sorted(sorted(range(n), key=key)[:budget])


def check_select(mass, lens, budget, sink, recent, err=0):
    K = kvx()
    R, H, W = mass.shape
    keep = torch.full((R + 2, H, budget), 99, dtype=torch.int32, device=DEV)
    new = torch.full((R + 2,), 99, dtype=torch.int64, device=DEV)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    K.kvx_evict_select(mass.to(DEV), torch.tensor(lens, device=DEV), budget, sink, recent, keep[1:R + 1], new[1:R + 1], flag)
    torch.cuda.synchronize()
    assert int(flag.item()) == err
    assert bool((keep[0] == 99).all()) and bool((keep[R + 1] == 99).all()) and new[0] == 99 and new[R + 1] == 99
    for r in range(R):
        n = min(max(lens[r], 0), W)
        assert int(new[r + 1]) == min(n, budget)
        for h in range(H):
            want = chosen(mass[r, h].numpy(), n, budget, sink, recent)
            got = keep[r + 1, h].tolist()
            assert got == want + [-1] * (budget - len(want)), (r, h)
    return keep[1:R + 1], new[1:R + 1]


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 1000, 1024, 1025, 5000, 40000])
def test_select_lengths(n):
    mass = torch.rand(2, 2, n, generator=torch.Generator().manual_seed(n)) ** 6
    for budget in sorted({1, 2, max(1, n // 3), max(1, n - 1), n, n + 3}):
        check_select(mass, [n, max(0, n - 7)], budget, 0, 0)
        if budget > 4:
            check_select(mass, [n, max(0, n - 7)], budget, 2, budget // 2)


@pytest.mark.parametrize("n", [1023, 16384, 16385, 32767, 32768, 32769, 65536, 70001])
def test_select_long_lists(n):
    """Around the slots that the registers hold at once, with ties across them and masses that share their leading bits."""
    g = torch.Generator().manual_seed(n)
    mass = torch.stack([torch.rand(n, generator=g) * 2.0 ** -20 + 1, torch.randint(0, 3, (n,), generator=g).float()])[None]
    for budget in (1, 700, n // 2, n - 1):
        check_select(mass, [n], budget, min(4, budget - 1), min(64, budget // 2))


def test_select_ties_and_special_values():
    g = torch.Generator().manual_seed(3)
    ties = torch.randint(0, 4, (3, 2, 3000), generator=g).float()
    ties[0, 0] = 0
    ties[0, 1, ::2] = -0.0
    check_select(ties, [3000, 2999, 100], 700, 4, 33)
    odd = torch.rand(1, 3, 2000, generator=g)
    odd[0, 0, ::3], odd[0, 0, 1::3] = math.nan, math.inf
    odd[0, 1, :] = -odd[0, 1, :]  # negative masses are ordered too
    odd[0, 1, 5] = -math.inf
    odd[0, 2, 100] = math.nan
    odd[0, 2, 200:900] = 1e-45  # denormal, equal
    check_select(odd, [2000], 1000, 3, 5)
    check_select(odd, [2000], 1, 1, 0)
    check_select(odd, [2000], 40, 0, 40)


def test_select_lengths_outside_the_masses():
    K = kvx()
    mass = torch.rand(4, 1, 300, generator=torch.Generator().manual_seed(4))
    check_select(mass, [300, 1 << 40, -3, 0], 50, 2, 10, err=K.DEVERR_TABLE_RANGE)


def test_select_strided():
    base = torch.rand(3, 4, 700, generator=torch.Generator().manual_seed(5)).to(DEV)
    K = kvx()
    view = base[:, 1:3, 50:650]
    keep, new = torch.empty(3, 2, 128, dtype=torch.int32, device=DEV), torch.empty(3, dtype=torch.int64, device=DEV)
    K.kvx_evict_select(view, torch.tensor([600, 128, 129], device=DEV), 128, 4, 20, keep, new)
    torch.cuda.synchronize()
    for r, n in enumerate((600, 128, 129)):
        for h in range(2):
            assert keep[r, h].tolist() == chosen(view[r, h].cpu().numpy(), n, 128, 4, 20)


def moved(case, keep, dst_table, mass, out_width):
    """The cache and masses after the move, on the host."""
    cache = case.cache.clone()
    src, dst = A.as_tokens(case.cache, case.layout), A.as_tokens(cache, case.layout)
    R, H, B = keep.shape
    out = torch.zeros(R, H, out_width)
    for r in range(R):
        for g in range(case.kv_heads):
            h = g // (case.kv_heads // H)
            for i in range(B):
                k = int(keep[r, h, i])
                if k < 0:
                    continue
                dst[int(dst_table[r, i // case.block]), i % case.block, :, g] = \
                    src[int(case.table[r, k // case.block]), k % case.block, :, g]
                if i < out_width:
                    out[r, h, i] = mass[r, h, k]
    return cache, out


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("lists", [1, 2, 4])
@pytest.mark.parametrize("dim,block,layout", [(128, 16, A.LAYOUTS[0]), (64, 16, A.LAYOUTS[2]), (40, 3, A.LAYOUTS[1]),
                                              (8, 1, A.LAYOUTS[0]), (256, 64, A.LAYOUTS[1]), (72, 24, A.LAYOUTS[2])])
def test_compact(in_place, lists, dim, block, layout):
    K = kvx()
    lens = [(1, 700), (1, 90), (1, 0), (1, 333)]
    case = A.Case(30, lens, heads=4, kv_heads=4, dim=dim, block=block, layout=layout, spare=160 if block > 3 else 620)
    B = 150
    mass = torch.rand(4, lists, 720, generator=torch.Generator().manual_seed(6)) ** 4
    keep, new = check_select(mass, [c for _, c in lens], B, 4, 16)
    dst = case.table.copy()
    if not in_place:
        free = np.setdiff1d(np.arange(case.num_blocks), case.table[case.table >= 0])
        cols = -(-B // block)
        dst = np.full((4, cols), -1, np.int32)
        at = 0
        for r in range(4):
            n = -(-int(new[r]) // block)
            dst[r, :n] = free[at:at + n]
            at += n
    width = 720 if in_place else 170
    want, want_mass = moved(case, keep.cpu(), dst, mass, width)
    cache, m = case.cache.to(DEV), mass.to(DEV)
    table = torch.from_numpy(case.table).to(DEV)
    to = table if in_place else torch.from_numpy(dst).to(DEV)
    out = m if in_place else torch.full((4, lists, 190), 5.0, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    K.kvx_evict_compact(cache, table, to, keep, m, out[:, :, :width], layout=layout, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert torch.equal(cache.cpu().view(torch.int16), want.view(torch.int16))
    assert torch.equal(out[:, :, :width].cpu(), want_mass)
    assert in_place or bool((out[:, :, width:] == 5).all())


def test_compact_in_place_at_length():
    """A long column moved in place through many tiles, without masses."""
    K = kvx()
    case = A.Case(31, [(1, 6000)], heads=2, kv_heads=2, dim=64, spare=0)
    mass = torch.rand(1, 2, 6000, generator=torch.Generator().manual_seed(7))
    mass[0, 0, :3000] += 1  # head 0 keeps its first half where it is
    mass[0, 1, 3000:] += 1  # head 1 moves its second half over the first
    keep, _ = check_select(mass, [6000], 3001, 0, 0)
    want, _ = moved(case, keep.cpu(), case.table, mass, 1)
    cache, table = case.cache.to(DEV), torch.from_numpy(case.table).to(DEV)
    K.kvx_evict_compact(cache, table, table, keep)
    torch.cuda.synchronize()
    assert torch.equal(cache.cpu().view(torch.int16), want.view(torch.int16))


def test_compact_bad_lists_and_tables():
    """Entries outside the tables or the cache, or below their own index, move nothing."""
    K = kvx()
    case = A.Case(32, [(1, 100), (1, 100)], heads=1, kv_heads=1, dim=64, spare=20)
    free = np.setdiff1d(np.arange(case.num_blocks), case.table)
    dst = free[:6].reshape(2, 3).astype(np.int32)
    keep = np.stack([np.arange(0, 80, 2), np.arange(5, 45)])[:, None].astype(np.int32)
    good = keep.copy()
    for at, x in (((0, 0, 7), 3), ((0, 0, 9), 112), ((1, 0, 30), 1 << 30), ((1, 0, 39), -1)):
        keep[at], good[at] = x, -1
    mass = torch.rand(2, 1, 100, generator=torch.Generator().manual_seed(8))
    want, want_mass = moved(case, good, dst, mass, 40)
    cache, out, err = case.cache.to(DEV), torch.full((2, 1, 40), 5.0, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    table = torch.from_numpy(case.table).to(DEV)
    K.kvx_evict_compact(cache, table, torch.from_numpy(dst).to(DEV), torch.from_numpy(keep).to(DEV), mass.to(DEV), out,
                        err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == K.DEVERR_OFFSETS | K.DEVERR_TABLE_RANGE
    assert torch.equal(cache.cpu().view(torch.int16), want.view(torch.int16)) and torch.equal(out.cpu(), want_mass)
    # blocks outside the cache on either side; a destination table too narrow for the budget
    t2, d2 = case.table.copy(), dst.copy()
    t2[0, 1], d2[1, 2] = case.num_blocks, -1
    g2 = good.copy()
    g2[0, 0, [i for i in range(40) if 16 <= good[0, 0, i] < 32]] = -1
    g2[1, 0, 32:] = -1
    want, _ = moved(case, g2, dst, mass, 40)
    cache, err = case.cache.to(DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    K.kvx_evict_compact(cache, torch.from_numpy(t2).to(DEV), torch.from_numpy(d2).to(DEV), torch.from_numpy(good).to(DEV),
                        err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == K.DEVERR_BLOCK_RANGE
    assert torch.equal(cache.cpu().view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
def test_serving_chain(graph):
    """A prompt chunk and decode steps through all calls, with an eviction in the middle, against the
    same chain in float64 on the host: the caches bit for bit where rows are only moved, the
    attention within its tolerance after every step."""
    K = kvx()
    R, H, Hk, D, bs, budget = 3, 8, 2, 64, 16, 96
    g = torch.Generator().manual_seed(40)
    lens = [180, 64, 131]
    width, nb = 16, 60
    case = A.Case(40, [(n, n) for n in lens], heads=H, kv_heads=Hk, dim=D, spare=nb - 25)
    case.width = width
    table = np.full((R, width), -1, np.int32)
    ids = np.random.default_rng(1).permutation(case.num_blocks)
    for r in range(R):
        table[r] = ids[r * width:(r + 1) * width]
    case.table = table
    case.cache.fill_(math.nan)
    freq = (1e4 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float().to(DEV)
    axis = [0] * (D // 2)
    dev_table, cache = torch.from_numpy(table).to(DEV), case.cache.to(DEV)
    mass = torch.zeros(R, Hk, width * bs, device=DEV)
    keep = torch.empty(R, Hk, budget, dtype=torch.int32, device=DEV)
    new_lens = torch.empty(R, dtype=torch.int64, device=DEV)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device=DEV)
    held = list(lens)  # tokens in the cache
    seen = list(lens)  # tokens so far: the next position

    def step(new):
        """One forward step's calls for `new` tokens a request; checks the attention."""
        T = sum(new)
        q, k, v = (torch.randn(T, n, D, generator=g).to(torch.bfloat16) for n in (H, Hk, Hk))
        off = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
        pos = torch.cat([torch.arange(seen[r] - new[r], seen[r]) for r in range(R)])[None].contiguous()
        slot = torch.cat([torch.arange(held[r] - new[r], held[r]) for r in range(R)]).to(DEV)
        req = torch.cat([torch.full((new[r],), r, dtype=torch.int32) for r in range(R)]).to(DEV)
        slots, out = torch.empty(T, dtype=torch.int64, device=DEV), torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV)
        qr, lse = torch.empty_like(out), torch.empty(T, H, device=DEV)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        dq, dk, dv, dpos, doff = q.to(DEV), k.to(DEV), v.to(DEV), pos.to(DEV), torch.from_numpy(off).to(DEV)
        ctx = torch.tensor(held, dtype=torch.int64, device=DEV)
        before = mass.clone()

        def calls():
            K.kvx_slot_mapping(dev_table, req, slot, bs, slots, err)
            K.kvx_rope_and_cache(dq, dk, dv, dpos, freq, axis, slots, cache, qr, err_flag=err)
            K.kvx_paged_attention(qr, cache, dev_table, doff, ctx, out, lse, workspace=ws, err_flag=err,
                                  max_query_len=max(new))
            K.kvx_attention_mass(qr, cache, dev_table, doff, ctx, lse, mass, err_flag=err)
        if graph:
            cg = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(cg):
                calls()
            for _ in range(2):
                mass.copy_(before)
                out.fill_(math.nan)
                torch.cuda.synchronize()
                cg.replay()
                torch.cuda.synchronize()
        else:
            calls()
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        case.lens, case.offsets, case.T = list(zip(new, held)), off, T
        case.context, case.q, case.cache = np.array(held, np.int64), qr.cpu(), cache.cpu()
        want, want_lse, tol, tol_lse = A.attention(case)
        A.check("out", out, want, tol)
        A.check("lse", lse, want_lse, tol_lse)
        added, tol_m, _ = A.masses(case, lse.cpu())
        total = before.cpu().double() + added
        A.check("mass", mass, total, tol_m + total * 2.0 ** -24)

    step(list(lens))
    for _ in range(2):
        for r in range(R):
            held[r] += 1
            seen[r] += 1
        step([1] * R)
    ctx = torch.tensor(held, dtype=torch.int64, device=DEV)
    case.context, case.cache, host_mass = np.array(held, np.int64), cache.cpu(), mass.cpu()
    K.kvx_evict_select(mass, ctx, budget, 4, 32, keep, new_lens)
    K.kvx_evict_compact(cache, dev_table, dev_table, keep, mass, mass)
    torch.cuda.synchronize()
    for r in range(R):
        for h in range(Hk):
            want = chosen(host_mass[r, h].numpy(), held[r], budget, 4, 32)
            assert keep[r, h].tolist() == want + [-1] * (budget - len(want))
    want, want_mass = moved(case, keep.cpu(), table, host_mass, width * bs)
    assert torch.equal(cache.cpu().view(torch.int16), want.view(torch.int16)) and torch.equal(mass.cpu(), want_mass)
    held = new_lens.tolist()
    for _ in range(2):
        for r in range(R):
            held[r] += 1
            seen[r] += 1
        step([1] * R)
