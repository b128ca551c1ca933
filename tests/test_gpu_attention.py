"""kvx_paged_attention and kvx_attention_mass against float64 results, at the sizes, masks and
layouts where they can go wrong."""
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


def run(case, causal=True, window=0, scale=None, err=0, split=True, mass=True):
    dev = case.to()
    want, want_lse, tol, tol_lse = A.attention(case, causal, window, scale)
    out, lse, bits = A.attend(case, dev, causal, window, scale, split)
    used = int(case.offsets[-1])
    assert bits == err
    A.check("out", out[:used], want[:used], tol[:used])
    A.check("lse", lse[:used], want_lse[:used], tol_lse[:used])
    assert bool((out[used:] == 7).all()) and bool((lse[used:] == 7).all()), "rows of nobody were written"
    if not mass:
        return
    added, tol_m, seen = A.masses(case, lse.cpu(), causal, window, scale)
    K = kvx()
    start = torch.rand(added.shape, generator=torch.Generator().manual_seed(1))
    m = start.to(DEV)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    K.kvx_attention_mass(dev[0], dev[1], dev[2], dev[3], dev[4], lse, m, scale=scale, causal=causal, window=window,
                         layout=case.layout, err_flag=flag)
    torch.cuda.synchronize()
    assert int(flag.item()) == err
    total = start.double() + added
    A.check("mass", m, total, tol_m + total.abs() * 2.0 ** -24)
    assert torch.equal(m.cpu()[~seen], start[~seen]), "slots no row sees were written"


# one token, few, many: below and across the tiles of 32 and 128 rows and of 32 and 64 slots
LENS = {
    "one": [(1, 1)], "two_slots": [(1, 2), (1, 31), (1, 32), (1, 33)], "decode": [(1, 129), (1, 1), (1, 700), (1, 64)],
    "drafted": [(4, 300), (3, 3), (5, 77), (1, 65)], "tile_edges": [(16, 63), (17, 64), (33, 65), (64, 128), (65, 129)],
    "prompts": [(97, 97), (1, 1), (128, 128), (129, 129)], "chunk": [(70, 513), (200, 1000)],
    "with_empty": [(0, 0), (3, 40), (0, 17), (2, 2), (0, 0)],
}


@pytest.mark.parametrize("lens", list(LENS), ids=list(LENS))
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_lengths(lens, dtype):
    run(A.Case(1, LENS[lens], heads=8, kv_heads=2, dim=128, dtype=dtype))


@pytest.mark.parametrize("dim", [8, 16, 40, 64, 72, 80, 96, 128, 136, 192, 256])
@pytest.mark.parametrize("lens", ["drafted", "tile_edges"])
def test_head_dims(dim, lens):
    run(A.Case(2, LENS[lens], heads=4, kv_heads=2, dim=dim, dtype="bf16" if dim % 16 else "fp16"))


@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 3), (5, 1), (7, 1), (14, 2), (32, 1), (33, 1), (40, 1), (128, 1), (130, 2)])
@pytest.mark.parametrize("lens", [[(1, 200), (1, 33)], [(6, 90), (1, 5), (19, 64)]], ids=["decode", "chunk"])
def test_head_groups(heads, kv, lens):
    run(A.Case(3, lens, heads=heads, kv_heads=kv, dim=64))


@pytest.mark.parametrize("layout", A.LAYOUTS)
@pytest.mark.parametrize("block", [1, 3, 16, 24, 64, 256])
def test_layouts_and_blocks(layout, block):
    run(A.Case(4, [(1, 170), (9, 130), (40, 257)], dim=64, block=block, layout=layout))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 7, 64, 100, 1 << 40])
@pytest.mark.parametrize("lens", [[(1, 500), (2, 64)], [(150, 400), (90, 90), (33, 321)]], ids=["decode", "chunk"])
def test_masks(causal, window, lens):
    run(A.Case(5, lens, dim=64), causal, window)


@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_see_nothing(causal):
    """More new tokens than context (the first ones see nothing), and no context at all."""
    case = A.Case(6, [(5, 2), (40, 7), (3, 0), (150, 70), (1, 0)], dim=64)
    run(case, causal)
    out, lse, _ = A.attend(case, case.to(), causal)
    assert bool((out[45:48] == 0).all()) and bool((lse[45:48] == -math.inf).all())


def test_rows_of_nobody_and_rows_behind():
    run(A.Case(7, [(3, 50), (40, 140)], dim=64, extra=37))
    run(A.Case(8, [(1, 50)], dim=64, extra=1))


def test_no_requests():
    K = kvx()
    q = torch.ones(4, 4, 64, dtype=torch.bfloat16, device=DEV)
    kv = torch.zeros(3, 16, 2, 2, 64, dtype=torch.bfloat16, device=DEV)
    none = torch.zeros(0, dtype=torch.int64, device=DEV)
    out = torch.full_like(q, 7)
    K.kvx_paged_attention(q, kv, torch.zeros(0, 3, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV),
                          none, out)
    K.kvx_paged_attention(q[:0], kv, torch.zeros(1, 3, dtype=torch.int32, device=DEV),
                          torch.zeros(2, dtype=torch.int64, device=DEV), torch.ones(1, dtype=torch.int64, device=DEV), out[:0])
    torch.cuda.synchronize()
    assert bool((out == 7).all())


@pytest.mark.parametrize("n", [1, 20, 140])
def test_unseen_slots_may_hold_anything(n):
    """A NaN or infinity in K or V reaches the rows that see it and no others."""
    case = A.Case(9, [(n, n + 150)], heads=4, kv_heads=2, dim=64)
    rows = A.as_tokens(case.cache, case.layout)
    for k, (slot, which, d, x) in enumerate([(n + 149, 1, 5, math.nan), (n + 140, 1, 17, math.inf), (n + 149, 0, 3, math.nan),
                                             (n + 100, 1, 40, -math.inf)]):
        if slot < 150 and n > 1:
            continue
        b, o = case.where(0, [slot])
        rows[b, o, which, k % 2, d] = x
    run(case, mass=False)
    run(case, window=60, mass=False)


def test_infinite_scores():
    """Scores of -inf weigh nothing; a row of nothing else counts as empty."""
    case = A.Case(10, [(2, 90)], heads=2, kv_heads=1, dim=64)
    rows = A.as_tokens(case.cache, case.layout)
    case.q[:, :, 0] = 1.0
    for slots in (range(3, 40), range(90)):
        b, o = case.where(0, list(slots))
        rows[b, o, 0, 0, 0] = -math.inf
        out, lse, bits = A.attend(case, case.to())
        if len(slots) == 90:
            assert bool((out == 0).all()) and bool((lse == -math.inf).all())
        else:
            want, want_lse, tol, tol_lse = A.attention(case)
            A.check("lse", lse, want_lse, tol_lse)
            A.check("out", out, want, tol)


def test_large_scores():
    """Scores of some thousands: the softmax picks one slot, and nothing overflows."""
    case = A.Case(11, [(1, 300), (30, 300)], dim=128, q_scale=200.0)
    run(case, mass=False)


@pytest.mark.parametrize("heads", [2, 8])
@pytest.mark.parametrize("lens", [[(1, 20011)], [(1, 9000), (1, 17), (1, 4097)], [(40, 12345)], [(130, 6001), (2, 40)]],
                         ids=["one", "ragged", "chunk", "mixed"])
def test_split_contexts(lens, heads):
    """Long contexts, with and without the workspace that splits them, give the same to rounding."""
    case = A.Case(12, lens, heads=heads, kv_heads=1, dim=128)
    run(case)
    run(case, split=False, mass=False)
    run(case, window=3000)


def test_many_requests():
    """More requests than a wavefront has lanes, empty ones among them: decode steps and chunks whose
    work is shared out, and a single head whose tiles are not."""
    rng = np.random.default_rng(12)
    lens = [(int(n), int(c)) if n else (0, int(c)) for n, c in zip(rng.integers(0, 2, 150), rng.integers(1, 900, 150))]
    run(A.Case(26, lens, heads=2, kv_heads=1, dim=64, extra=3))
    lens = [(int(n), int(n + c)) for n, c in zip(rng.integers(0, 60, 90), rng.integers(0, 600, 90))]
    run(A.Case(27, lens, heads=4, kv_heads=1, dim=64))
    run(A.Case(28, lens, heads=4, kv_heads=1, dim=64), split=False, mass=False)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_masses_of_a_large_batch(dim):
    """Enough slots to fill the GPU without splitting the rows: 5 heads a KV head, some windows."""
    case = A.Case(29, [(8, 1100)] * 14 + [(9, 700), (7, 2000)], heads=40 if dim == 64 else 32, kv_heads=8, dim=dim)
    run(case, window=0 if dim == 64 else 600)


@pytest.mark.parametrize("heads,kv,dim", [(33, 1, 64), (14, 2, 128), (3, 1, 136)])
@pytest.mark.parametrize("causal", [True, False])
def test_masses_of_head_groups(heads, kv, dim, causal):
    """Groups that the tiles of 32 rows do not divide, over many tiles, in the same launch as short requests."""
    run(A.Case(36, [(60, 900)] * (150 // kv) + [(97, 97), (11, 1000)], heads=heads, kv_heads=kv, dim=dim, extra=2), causal=causal,
        window=333 if causal else 0)


@pytest.mark.parametrize("dim,dtype", [(80, "bf16"), (256, "fp16")])
def test_shared_work_of_other_dims(dim, dtype):
    run(A.Case(30, [(1, 6000), (1, 200), (1, 3001)], heads=4, kv_heads=1, dim=dim, dtype=dtype))
    run(A.Case(31, [(70, 3000), (3, 900)], heads=4, kv_heads=1, dim=dim, dtype=dtype, block=24))


def test_every_workspace_size():
    """Any workspace from none to the full one is enough for right results."""
    K = kvx()
    case = A.Case(13, [(1, 5000), (1, 300)], heads=8, kv_heads=1, dim=64)
    q, cache, table, off, ctx = case.to()
    want, want_lse, tol, tol_lse = A.attention(case)
    full = K.attention_workspace_bytes(q, cache, 2, 1, 5000)
    guard = 4096
    for n in sorted({0, 1, 16, full // 7, full // 3, max(full - 1, 0), full, full + 4096}):
        buf = torch.full((n + guard,), 0xA5, dtype=torch.uint8, device=DEV)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
        K.kvx_paged_attention(q, cache, table, off, ctx, out, lse, workspace=buf[:n] if n else None, max_query_len=1,
                              max_context_len=5000)
        torch.cuda.synchronize()
        A.check("out", out, want, tol)
        A.check("lse", lse, want_lse, tol_lse)
        assert bool((buf[n:] == 0xA5).all()), "written past the workspace"


@pytest.mark.parametrize("hint", [(1, 1), (1, 1 << 20), (1 << 20, 1), (64, 64)])
def test_hints_are_only_hints(hint):
    K = kvx()
    case = A.Case(14, [(90, 700), (1, 3000), (7, 7)], heads=8, kv_heads=2, dim=64)
    q, cache, table, off, ctx = case.to()
    want, want_lse, tol, tol_lse = A.attention(case)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    K.kvx_paged_attention(q, cache, table, off, ctx, out, lse, workspace=ws, max_query_len=hint[0], max_context_len=hint[1])
    m = torch.zeros(3, 2, case.width * 16, device=DEV)
    K.kvx_attention_mass(q, cache, table, off, ctx, lse, m, max_query_len=hint[0], max_context_len=hint[1])
    torch.cuda.synchronize()
    A.check("out", out, want, tol)
    A.check("lse", lse, want_lse, tol_lse)
    added, tol_m, _ = A.masses(case, lse.cpu())
    A.check("mass", m, added, tol_m)


@pytest.mark.parametrize("n", [1, 50])
def test_strided_tensors(n):
    """Query and output as slices of wider tensors, a head-major cache, a table that is a slice."""
    K = kvx()
    case = A.Case(15, [(n, 200), (n, 333)], heads=6, kv_heads=2, dim=64)
    q, cache, table, off, ctx = case.to()
    T = q.shape[0]
    wide = torch.full((T, 6 + 4, 3 * 64), 3.0, dtype=q.dtype, device=DEV)
    wide[:, 2:8, 64:128] = q
    outs = torch.full((6, T + 2, 72), 7.0, dtype=q.dtype, device=DEV)  # head-major, rows 144 bytes apart
    head_major = cache.permute(0, 2, 3, 1, 4).contiguous()  # [blocks][K, V][heads][tokens][dim]
    view = head_major.permute(0, 1, 3, 2, 4)
    tables = torch.full((2, case.width + 5), -1, dtype=torch.int32, device=DEV)
    tables[:, :case.width] = table
    want, want_lse, tol, tol_lse = A.attention(case)
    out, lse = outs[:, 1:T + 1, :64].transpose(0, 1), torch.empty(T, 6, device=DEV)
    K.kvx_paged_attention(wide[:, 2:8, 64:128], view, tables[:, :case.width], off, ctx, out, lse, layout=A.LAYOUTS[1])
    m = torch.zeros(2, 2, 777, device=DEV)
    K.kvx_attention_mass(wide[:, 2:8, 64:128], view, tables[:, :case.width], off, ctx, lse, m[:, :, 5:5 + 500],
                         layout=A.LAYOUTS[1])
    torch.cuda.synchronize()
    A.check("out", out, want, tol)
    A.check("lse", lse, want_lse, tol_lse)
    assert bool((outs[:, 0] == 7).all()) and bool((outs[:, T + 1] == 7).all()) and bool((outs[..., 64:] == 7).all())
    added, tol_m, _ = A.masses(case, lse.cpu())
    w = added.shape[2]
    A.check("mass", m[:, :, 5:5 + w], added, tol_m)
    assert bool((m[:, :, :5] == 0).all()) and bool((m[:, :, 5 + w:] == 0).all())


def test_offsets_past_32_bits():
    """Blocks 3 GiB apart in one cache: a row's byte offset passes 2^32."""
    K = kvx()
    case = A.Case(16, [(1, 70), (20, 66)], heads=4, kv_heads=1, dim=64)
    q, cache, table, off, ctx = case.to()
    far = 3 << 29  # elements
    big = torch.empty(far * (case.num_blocks - 1) + 4096, dtype=torch.bfloat16, device=DEV)
    view = torch.as_strided(big, (case.num_blocks, 16, 2, 1, 64), (far, 128, 64, 64, 1))
    for b in range(case.num_blocks):
        view[b].copy_(cache[b])
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
    K.kvx_paged_attention(q, view, table, off, ctx, out, lse)
    m = torch.zeros(2, 1, case.width * 16, device=DEV)
    K.kvx_attention_mass(q, view, table, off, ctx, lse, m)
    torch.cuda.synchronize()
    want, want_lse, tol, tol_lse = A.attention(case)
    A.check("out", out, want, tol)
    added, tol_m, _ = A.masses(case, lse.cpu())
    A.check("mass", m, added, tol_m)


@pytest.mark.parametrize("n", [1, 20, 100])
def test_bad_tables(n):
    """Entries outside the cache are slots not seen, and raise their bit; so do contexts longer
    than the table's row, which are cut there, and negative ones."""
    K = kvx()
    case = A.Case(17, [(n, n + 200), (n, 150), (1, 40)], heads=4, kv_heads=2, dim=64)
    case.table[0, 3], case.table[0, 5], case.table[1, 0] = -1, case.num_blocks, 1 << 30
    run(case, err=K.DEVERR_BLOCK_RANGE)
    case = A.Case(18, [(n, n + 200), (n, n + 64)], heads=4, kv_heads=2, dim=64)
    case.context[0] = 1 << 40
    case.table[0, :] = case.table[0, 0]  # every column a block of the cache
    case.table[1, case.table[1] < 0] = 0
    rows = A.as_tokens(case.cache, case.layout)
    rows[rows.isnan()] = 0.5
    run(case, err=K.DEVERR_TABLE_RANGE)
    case = A.Case(19, [(n, n + 20), (n, n + 64)], heads=4, kv_heads=2, dim=64)
    case.context[0] = -5
    run(case, err=K.DEVERR_TABLE_RANGE)


@pytest.mark.parametrize("offsets", [[0, 50, 20, 60], [0, 10, 70, 1 << 40], [-3, 10, 20, 60], [55, 10, 20, 60], [60, 0, 60, 0],
                                     [0, 60, 0, 60], [0, -5, 60, 61]])
@pytest.mark.parametrize("split", [False, True])
def test_bad_offsets(offsets, split):
    """Offsets that are not a CSR raise their bit and reach nothing outside the tensors, among them
    ones that give the same rows to several requests."""
    K = kvx()
    for heads, ctx_len in ((4, 60), (64, 3000)):
        case = A.Case(20, [(20, ctx_len), (20, 60), (20, ctx_len)], heads=heads, kv_heads=2, dim=64)
        q, cache, table, _, ctx = case.to()
        off = torch.tensor(offsets, dtype=torch.int64, device=DEV)
        guard = torch.full((62, heads, 64), 7.0, dtype=q.dtype, device=DEV)
        err = torch.zeros(2, dtype=torch.int32, device=DEV)
        lses = torch.full((62, heads), 7.0, device=DEV)
        n = K.attention_workspace_bytes(q, cache, 3, 20, ctx_len) if split else 0
        ws = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
        K.kvx_paged_attention(q, cache, table, off, ctx, guard[1:61], lses[1:61], err_flag=err[:1], max_query_len=20,
                              max_context_len=ctx_len, workspace=ws[:n] if n else None)
        m = torch.zeros(3, 2, case.width * 16, device=DEV)
        K.kvx_attention_mass(q, cache, table, off, ctx, torch.zeros(60, heads, device=DEV), m, err_flag=err[1:])
        torch.cuda.synchronize()
        assert err.tolist() == [K.DEVERR_OFFSETS] * 2
        for t in (guard, lses):
            assert bool((t[0] == 7).all()) and bool((t[61] == 7).all())
        assert bool((ws[n:] == 0xA5).all()), "written past the workspace"


def test_narrow_masses():
    """Masses narrower than a context are cut there and raise the bit."""
    K = kvx()
    case = A.Case(21, [(3, 90), (1, 40)], heads=4, kv_heads=2, dim=64)
    q, cache, table, off, ctx = case.to()
    out, lse, _ = A.attend(case, (q, cache, table, off, ctx))
    m = torch.zeros(2, 2, 80, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    K.kvx_attention_mass(q, cache, table, off, ctx, lse, m[:, :, :70], err_flag=err)
    torch.cuda.synchronize()
    added, tol, _ = A.masses(case, lse.cpu())
    assert int(err.item()) == K.DEVERR_TABLE_RANGE
    A.check("mass", m[:, :, :70], added[:, :, :70], tol[:, :, :70])
    assert bool((m[:, :, 70:] == 0).all())


def test_the_same_bits_every_time():
    K = kvx()
    case = A.Case(22, [(1, 9000), (50, 400), (3, 3)], heads=8, kv_heads=2, dim=128)
    dev = case.to()
    first = A.attend(case, dev)
    ms = []
    for _ in range(3):
        again = A.attend(case, dev)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
        m = torch.zeros(3, 2, case.width * 16, device=DEV)
        K.kvx_attention_mass(*dev, first[1], m)
        ms.append(m)
    torch.cuda.synchronize()
    assert torch.equal(ms[0], ms[1]) and torch.equal(ms[0], ms[2])


def test_two_streams_and_captured_graphs():
    """Two batches at once on two streams, each with its workspace, and both captured and replayed
    with eager work between the replays."""
    K = kvx()
    cases = [A.Case(23, [(1, 6000), (1, 50)], heads=8, kv_heads=1, dim=128), A.Case(24, [(60, 3000)], heads=8, kv_heads=2, dim=64)]
    state = []
    for case in cases:
        q, cache, table, off, ctx = dev = case.to()
        n, c = max(x for x, _ in case.lens), int(case.context.max())
        ws = K.new_attention_workspace(q, cache, len(case.lens), n, c)
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device=DEV)
        m = torch.zeros(len(case.lens), case.kv_heads, case.width * 16, device=DEV)

        def call(dev=dev, ws=ws, out=out, lse=lse, m=m, n=n, c=c):
            K.kvx_paged_attention(*dev, out, lse, workspace=ws, max_query_len=n, max_context_len=c)
            m.zero_()
            K.kvx_attention_mass(*dev, lse, m, max_query_len=n, max_context_len=c)

        state.append((case, dev, out, lse, m, call))
    streams = [torch.cuda.Stream() for _ in state]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, x in zip(streams, state):
            with torch.cuda.stream(s):
                x[5]()
    torch.cuda.synchronize()
    expect = []
    for case, dev, out, lse, m, _ in state:
        want, want_lse, tol, tol_lse = A.attention(case)
        A.check("out", out, want, tol)
        A.check("lse", lse, want_lse, tol_lse)
        added, tol_m, _ = A.masses(case, lse.cpu())
        A.check("mass", m, added, tol_m)
        expect.append((out.clone(), lse.clone(), m.clone()))
    graphs = []
    for x in state:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x[5]()
        graphs.append(g)
    for rep in range(3):
        for x in state:  # eager work between the replays: wipe the outputs
            for t in x[2:5]:
                t.fill_(math.nan)
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for x, e in zip(state, expect):
            assert all(torch.equal(a, b) for a, b in zip(x[2:5], e)), f"replay {rep}"
    # the graphs read lengths from the device: a longer context needs no new capture
    case, dev = state[0][0], state[0][1]
    dev[4].copy_(torch.tensor([5000, 33]))
    graphs[0].replay()
    torch.cuda.synchronize()
    case.context = np.array([5000, 33], np.int64)
    want, _, tol, _ = A.attention(case)
    A.check("out", state[0][2], want, tol)
