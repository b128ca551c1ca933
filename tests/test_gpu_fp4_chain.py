"""The calls on a 4-bit cache together, as a serving loop makes them: new rows appended, attention over them, whole blocks and head
shards transferred; eagerly, on another stream, from captured graphs, and two at a time."""
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


class Server:
    """Requests of some lengths on a 4-bit cache of one layer: tables, positions and inputs on the device."""

    def __init__(self, seed, lens, heads=8, kv=2, dim=64, block=16, dtype="bf16"):
        K, self.lens, self.dt = kvx(), list(lens), A.DT[dtype]
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        counts = [-(-n // block) for n in lens]
        self.heads, self.kv, self.dim, self.block, self.T, nb = heads, kv, dim, block, sum(lens), sum(counts) + 3
        ids = rng.permutation(nb).astype(np.int32)
        self.table_h = np.full((len(lens), max(counts)), -1, np.int32)
        for r, n in enumerate(counts):
            self.table_h[r, :n] = ids[sum(counts[:r]):sum(counts[:r]) + n]
        place = np.concatenate([np.arange(n) for n in lens])
        req = np.repeat(np.arange(len(lens)), lens)
        slots = self.table_h[req, place // block].astype(np.int64) * block + place % block

        def dev(x):
            return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)

        self.table, self.slots, self.pos = dev(self.table_h), dev(slots), dev(place.astype(np.int64)[None])
        self.offsets = dev(np.concatenate([[0], np.cumsum(lens)]).astype(np.int64))
        self.context = dev(np.array(lens, np.int64))
        self.q, self.k, self.v = (torch.randn((self.T, n, dim), generator=g).to(self.dt).to(DEV) for n in (heads, kv, kv))
        self.freq = (1e4 ** (-torch.arange(dim // 2, dtype=torch.float64) / (dim // 2))).float().to(DEV)
        self.axis = [0] * (dim // 2)
        self.cache = K.new_fp4_cache(nb, block, kv, dim, DEV)
        self.qr, self.out, self.ko, self.vo = torch.empty_like(self.q), torch.empty_like(self.q), torch.empty_like(self.k), torch.empty_like(self.v)
        self.lse = torch.empty(self.T, heads, device=DEV)
        self.ws = K.new_attention_workspace_fp4(self.q, self.cache, len(lens), max(lens), max(lens))

    def append(self, cache=None, **kw):
        kvx().kvx_rope_and_cache_fp4(self.q, self.k, self.v, self.pos, self.freq, self.axis, self.slots,
                                     self.cache if cache is None else cache, self.qr, self.ko, self.vo, **kw)

    def attend(self, cache=None, table=None, **kw):
        kvx().kvx_paged_attention_fp4(self.qr, self.cache if cache is None else cache, self.table if table is None else table, self.offsets,
                                      self.context, self.out, self.lse, workspace=self.ws, max_query_len=max(self.lens),
                                      max_context_len=max(self.lens), **kw)

    def check(self):
        """Attention of the rotated queries over what key_out and value_out say that the cache holds."""
        torch.cuda.synchronize()
        case = F.Case4(1, [(n, n) for n in self.lens], self.heads, self.kv, self.dim, self.block, "bf16" if self.dt == torch.bfloat16 else "fp16")
        case.q, held, at = self.qr.cpu(), torch.stack([self.ko, self.vo], 1).cpu().double(), np.concatenate([[0], np.cumsum(self.lens)])
        case.rows_of = lambda r: (held[at[r]:at[r + 1]], torch.ones(self.lens[r], dtype=torch.bool))
        want, want_lse, tol, tol_lse = F.attention(case)
        A.check("out", self.out, want, tol)
        A.check("lse", self.lse, want_lse, tol_lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("lens,dim,block", [([1], 64, 16), ([40, 7, 130], 64, 16), ([3, 33], 128, 24), ([200, 90], 256, 16)])
def test_append_and_attend(lens, dim, block, dtype):
    s = Server(1, lens, dim=dim, block=block, dtype=dtype)
    s.append()
    s.attend()
    s.check()


def test_prompt_then_single_tokens():
    """A prompt in one call, then tokens one by one: each step's attention sees all rows before it, and the cache ends with the
    bytes that one call for all tokens leaves."""
    K, s = kvx(), Server(2, [45])
    s.append()
    s.attend()
    torch.cuda.synchronize()
    whole, out, step = s.cache.clone(), s.out.clone(), K.new_fp4_cache(s.cache.shape[0], 16, 2, 64, DEV)
    n = 30
    for a, b in [(0, n)] + [(i, i + 1) for i in range(n, 45)]:
        qr = torch.empty_like(s.q[a:b])
        K.kvx_rope_and_cache_fp4(s.q[a:b], s.k[a:b], s.v[a:b], s.pos[:, a:b].contiguous(), s.freq, s.axis, s.slots[a:b], step, qr)
        got = torch.empty_like(qr)
        K.kvx_paged_attention_fp4(qr, step, s.table, torch.tensor([0, b - a], device=DEV), torch.tensor([b], device=DEV), got,
                                  max_query_len=b - a, max_context_len=b)
        torch.cuda.synchronize()
        # each call is within one rounding of its weights and one of the result, 2^-8 of max|v| each, of the same 64-bit
        # result (sums and scores of 45 slots add less than 1e-3): they differ by at most twice that
        assert float((got.float() - out[a:b].float()).abs().max()) <= 4 * 2.0 ** -8 * float(s.vo.float().abs().max()) + 1e-3
    assert torch.equal(step, whole)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_a_16_bit_cache_and_the_same_blocks_in_4_bits(dtype):
    """Rows rotated into a 16-bit cache and packed in 4 bits, received as a 4-bit cache and as a 16-bit one: the first attention
    equals the second's within both calls' bounds, and the 4-bit blocks are those of the format."""
    K, s = kvx(), Server(3, [50, 120], dtype=dtype)
    nb = s.cache.shape[0]
    wide, back = (torch.zeros(nb, 16, 2, s.kv, s.dim, dtype=s.dt, device=DEV) for _ in range(2))
    K.kvx_rope_and_cache(s.q, s.k, s.v, s.pos, s.freq, s.axis, s.slots, wide, s.qr)
    used = s.table_h[s.table_h >= 0]
    ids = torch.from_numpy(used).to(DEV)
    off = torch.tensor([0, len(used)], device=DEV)
    runs, count = K.new_xfer_list(len(used), DEV)
    to, to_count = K.new_xfer_list(len(used), DEV)
    K.kvx_build_xfer_list(ids, None, off, K.MODE_PACK, runs, count)
    K.kvx_build_xfer_list(None, ids, off, K.MODE_UNPACK, to, to_count)
    buf = K.new_fp4_cache(len(used), 16, s.kv, s.dim, DEV)
    K.kvx_pack_fp4(K.layer_base_table([wide]), wide, runs, count, len(used), buf)
    K.kvx_unpack([buf], K.layer_base_table([s.cache]), s.cache[0].numel(), nb, 1, to, to_count, len(used))
    K.kvx_unpack_fp4(buf, K.layer_base_table([back]), back, to, to_count, len(used))
    torch.cuda.synchronize()
    codes, scales = F.quantise(wide.double().cpu().numpy().transpose(0, 3, 2, 1, 4), F.MOST[s.dt])
    assert np.array_equal(s.cache.cpu().numpy()[used], F.to_planes(codes, scales)[used])
    held = torch.from_numpy(F.values(codes, scales).transpose(0, 3, 2, 1, 4)).to(s.dt)
    assert torch.equal(back.cpu()[used], held[used])
    s.ko, s.vo = (back.view(-1, 2, s.kv, s.dim)[s.slots, w] for w in (0, 1))
    s.attend()
    s.check()
    out, lse = torch.empty_like(s.out), torch.empty_like(s.lse)
    K.kvx_paged_attention(s.qr, back, s.table, s.offsets, s.context, out, lse, max_query_len=120, max_context_len=120)
    s.out, s.lse = out, lse
    s.check()


def test_transfer_of_a_4_bit_cache_whole_and_by_heads():
    """Its blocks are byte ranges: packed and unpacked to other ids they give the same attention, bit for bit; split by heads, each
    shard is a cache of its heads."""
    K, s = kvx(), Server(4, [70, 33], heads=8, kv=4)
    s.append()
    s.attend()
    torch.cuda.synchronize()
    out, lse = s.out.clone(), s.lse.clone()
    used = s.table_h[s.table_h >= 0]
    nb, bb, N = s.cache.shape[0], s.cache[0].numel(), len(used)
    new_ids = np.random.default_rng(5).permutation(nb + 5)[:N].astype(np.int32)
    ids, off = torch.from_numpy(used).to(DEV), torch.tensor([0, N], device=DEV)
    runs, count = K.new_xfer_list(N, DEV)
    K.kvx_build_xfer_list(ids, None, off, K.MODE_PACK, runs, count)
    to, to_count = K.new_xfer_list(N, DEV)
    K.kvx_build_xfer_list(None, torch.from_numpy(new_ids).to(DEV), off, K.MODE_UNPACK, to, to_count)
    buf = torch.empty(N * bb, dtype=torch.uint8, device=DEV)
    K.kvx_pack(K.layer_base_table([s.cache]), bb, nb, runs, count, N, buf)
    other = K.new_fp4_cache(nb + 5, 16, 4, 64, DEV)
    K.kvx_unpack([buf], K.layer_base_table([other]), bb, nb + 5, 1, to, to_count, N)
    table = s.table_h.copy()
    table[s.table_h >= 0] = new_ids
    s.attend(other, torch.from_numpy(table).to(DEV))
    torch.cuda.synchronize()
    assert torch.equal(s.out, out) and torch.equal(s.lse, lse)
    shards = [torch.empty(N * bb // 2, dtype=torch.uint8, device=DEV) for _ in range(2)]
    K.kvx_pack_split(K.layer_base_table([s.cache]), bb, nb, 1, runs, count, N, shards)
    order = np.full_like(s.table_h, -1)
    order[s.table_h >= 0] = np.arange(N)
    for d, shard in enumerate(shards):
        got = torch.empty(s.T, 4, 64, dtype=s.dt, device=DEV)
        K.kvx_paged_attention_fp4(s.qr[:, 4 * d:4 * d + 4], shard.view(N, 2, 2, -1), torch.from_numpy(order).to(DEV), s.offsets, s.context, got,
                                  max_query_len=70, max_context_len=70)
        torch.cuda.synchronize()
        assert torch.equal(got, out[:, 4 * d:4 * d + 4])
    merged = K.new_fp4_cache(nb + 5, 16, 4, 64, DEV)
    K.kvx_unpack(shards, K.layer_base_table([merged]), bb, nb + 5, 1, to, to_count, N)
    torch.cuda.synchronize()
    assert torch.equal(merged, other)


def step(s, wide, back, buf, runs, to, N):
    """Append, attend, and send the request's 16-bit blocks in 4 bits: what a graph captures."""
    K = kvx()
    s.append()
    s.attend()
    K.kvx_pack_fp4(s.bases, wide, *runs, N, buf)
    K.kvx_unpack_fp4(buf, s.back_bases, back, *to, N)


def graph_parts(seed, lens):
    K, s = kvx(), Server(seed, lens, heads=8, kv=1, dim=128)
    nb = s.cache.shape[0]
    wide = torch.randn(nb, 16, 2, 1, 128, device=DEV).to(s.dt)
    back = torch.zeros_like(wide)
    used = s.table_h[s.table_h >= 0]
    ids, off, N = torch.from_numpy(used).to(DEV), torch.tensor([0, len(used)], device=DEV), len(used)
    runs, to = K.new_xfer_list(N, DEV), K.new_xfer_list(N, DEV)
    K.kvx_build_xfer_list(ids, None, off, K.MODE_PACK, *runs)
    K.kvx_build_xfer_list(None, ids, off, K.MODE_UNPACK, *to)
    s.bases, s.back_bases = K.layer_base_table([wide]), K.layer_base_table([back])
    buf = K.new_fp4_cache(N, 16, 1, 128, DEV)
    return s, (wide, back, buf, runs, to, N)


def snapshot(s, parts):
    return [t.clone() for t in (s.cache, s.qr, s.ko, s.vo, s.out, s.lse, parts[1], parts[2])]


def test_replayed_graphs_with_eager_work_between():
    """Two captured steps with a workspace each, replayed in turn with new inputs, eager calls and synchronisations between."""
    made = []
    for seed, lens in ((6, [300, 40, 1]), (7, [900])):
        s, parts = graph_parts(seed, lens)
        step(s, *parts)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(s, *parts)
        made.append((s, parts, graph))
    for turn in range(4):
        for s, parts, graph in made:
            for t in (s.q, s.k, s.v, parts[0]):
                t.copy_(torch.randn(t.shape, device=DEV).to(t.dtype))
            step(s, *parts)
            torch.cuda.synchronize()
            want = snapshot(s, parts)
            for t in (s.cache, s.qr, s.ko, s.vo, s.out, s.lse, parts[1], parts[2]):
                t.zero_()
            torch.ones(1000, device=DEV).sum().item()
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(snapshot(s, parts), want):
                assert torch.equal(a, b), turn
    for s, _, _ in made:
        s.check()


def test_other_streams_side_by_side():
    """Two batches on two streams of their own at once, each with its workspace, give what they give alone."""
    both = [graph_parts(8, [700, 20]), graph_parts(9, [64, 1, 513])]
    want = []
    for s, parts in both:
        step(s, *parts)
        torch.cuda.synchronize()
        want.append(snapshot(s, parts))
        for t in (s.cache, s.qr, s.ko, s.vo, s.out, s.lse, parts[1], parts[2]):
            t.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in both]
    for _ in range(5):
        for (s, parts), stream in zip(both, streams):
            with torch.cuda.stream(stream):
                step(s, *parts)
    torch.cuda.synchronize()
    for (s, parts), w in zip(both, want):
        for a, b in zip(snapshot(s, parts), w):
            assert torch.equal(a, b)
    # a stream passed to the call
    s, parts = both[0]
    s.out.zero_()
    torch.cuda.synchronize()
    s.attend(stream=streams[1])
    streams[1].synchronize()
    assert torch.equal(s.out, want[0][4])
