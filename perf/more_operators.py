"""Cases, inputs, plain forms and 64-bit results of the operators on a paged KV cache that is held in 4 bits:

  append    rotary positions, and the write of the rotated K rows and the V rows into the cache, quantised on the way
  attend    attention of each request's new tokens (one, a few drafted ones, or a chunk) over its cache
  transfer  the listed blocks of every 16-bit layer quantised into a send buffer, and that buffer into the receiver's 16-bit blocks
  restore   blocks kept in 4 bits written back into 16-bit caches

An element is one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign (codes 0 to 7, and 8 more where negative), two to a byte, the
even one in the low half. 32 neighbouring elements of a row share a power of two 2^(s - 127), s a byte: the smallest with
which the largest of them stays below 7, and at most what keeps 6 times it finite in the 16-bit type. A block holds for
each head and for K and V its tokens' elements and then their scales.

`run` computes a case in elementary torch operations, or with `own` set through the library's entry points.
Lengths follow from a case alone, the contents of the tensors from the seed.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
MOST = {"bf16": 125, "fp16": 13}  # largest exponent of a scale
LAYOUTS = ("blocks_tokens_kv", "blocks_kv_tokens", "kv_blocks_tokens")  # of a 16-bit cache
LAYOUTS4 = ("blocks_heads_kv", "blocks_kv_heads", "kv_blocks_heads")    # of a 4-bit one


# ----------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------

def _case(op, name=None, **kw):
    c = {"op": op, "reqs": 1, "new": 1, "ctx": 1, "heads": 8, "kv_heads": 1, "dim": 128, "block": 16, "dtype": "bf16",
         "layout": 0, "salt": 0}
    if op == "append":
        c.update(axes=1, rot=128, interleaved=False)
    if op == "attend":
        c.update(causal=True, window=0)
    if op in ("transfer", "restore"):
        c.update(layers=1, run=16)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one decode step of a serving batch: rotate 32 tokens and write their rows; latency counts
        _case("append", "append_decode", reqs=32, ctx=8192, heads=32, kv_heads=8, salt=1),
        # a prefill of video tokens (time, height, width), 32 query and 8 KV heads
        _case("append", "append_prefill", reqs=4, new=4096, ctx=4096, heads=32, kv_heads=8, axes=3, salt=2),
        # the smallest decode: one request a few blocks long
        _case("attend", "attend_decode_small", ctx=129, salt=3),
        # a serving batch in decode: 32 requests of ragged lengths, 32 query and 8 KV heads
        _case("attend", "attend_decode_batch", reqs=32, ctx=8192, heads=32, kv_heads=8, salt=4),
        # decode of two long documents, K plane before V plane
        _case("attend", "attend_decode_long", reqs=2, ctx=131071, heads=32, kv_heads=8, dtype="fp16", layout=2, salt=5),
        # up to 4 drafted tokens of each request, 7 query heads a KV head, a sliding window, blocks of 24
        _case("attend", "attend_drafts_window", reqs=13, new=4, ctx=5003, heads=28, kv_heads=4, dim=96, dtype="fp16", block=24,
              layout=1, window=1024, salt=6),
        # 8 requests of 576 blocks, each with a chunk of new tokens, one KV head (an 8-way head shard)
        _case("attend", "attend_chunk_shard", reqs=8, new=517, ctx=9216, salt=7),
        # the chunk of a long prompt: 2048 new tokens behind the cached ones
        _case("attend", "attend_chunk_long", new=2048, ctx=32768, heads=32, kv_heads=8, salt=8),
        # two layers of three short requests
        _case("transfer", "transfer_small", layers=2, reqs=3, ctx=640, run=2, salt=9),
        # 48 layers of 8 requests x 576 blocks of 8 KiB, runs of 64 blocks
        _case("transfer", "transfer_layers", layers=48, reqs=8, ctx=9216, run=64, salt=10),
        # one layer's shared prefix of one request, 8 heads
        _case("restore", "restore_prefix", ctx=2047, kv_heads=8, dim=64, dtype="fp16", layout=1, run=4, salt=11),
        # 32 layers of 16 requests x 256 blocks at 4 heads, runs of 2 blocks
        _case("restore", "restore_layers", layers=32, reqs=16, ctx=4096, kv_heads=4, layout=2, run=2, salt=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "transfer", "restore"])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 7, 8])
    dim = rng.choice([64, 64, 96, 128, 128, 128, 192, 256])
    c = _case(op, reqs=_log_int(rng, 1, 48), heads=heads, kv_heads=kv_heads, dim=dim, block=rng.choice([16, 16, 16, 32, 64, 8, 24]),
              dtype=rng.choice(["bf16", "bf16", "fp16"]), layout=rng.randrange(3), salt=rng.randrange(1 << 30))
    if op == "append":
        c["new"] = _log_int(rng, 1, 4096)
        c["ctx"] = c["new"] + _log_int(rng, 1, 8192)
        c["axes"] = rng.choice([1, 2, 3, 4])
        c["rot"] = rng.choice([dim, dim, dim // 32 * 16])
        c["interleaved"] = rng.random() < 0.3
    elif op == "attend":
        c["new"] = rng.choice([1, 1, _log_int(rng, 2, 2048), _log_int(rng, 2, 128)])
        c["ctx"] = c["new"] + _log_int(rng, 1, 131072 if rng.random() < 0.3 else 16384)
        c["window"] = rng.choice([0, 0, 0, _log_int(rng, 16, 4096)])
        c["causal"] = rng.random() < 0.85
    else:
        c["ctx"] = _log_int(rng, 17, 16384)
        c["layers"] = _log_int(rng, 1, 48)
        c["run"] = _log_int(rng, 1, 64)
    most = {"append": "append_prefill", "attend": "attend_chunk_long", "transfer": "transfer_layers", "restore": "restore_layers"}[op]
    top = work(next(x for x in listed() if x["name"] == most))
    # a drawn case costs no more than the largest of its kind, in work and in the plain form's scores
    while work(c)["bytes"] > max(top["bytes"], 3e8) or (op == "attend" and (work(c)["flops"] > top["flops"] or
                                                        c["reqs"] * c["heads"] * c["new"] * c["ctx"] > 2.2e9)):
        if c["reqs"] > 1:
            c["reqs"] = (c["reqs"] + 1) // 2
        elif c.get("layers", 1) > 1:
            c["layers"] = (c["layers"] + 1) // 2
        elif c["new"] > 64:
            c["ctx"] -= c["new"] // 2
            c["new"] -= c["new"] // 2
        else:
            c["ctx"] = max(c["new"], c["ctx"] * 2 // 3)
    return c


def _lengths(c):
    """(new tokens, context with them) of every request; the first request has the case's own."""
    rng = random.Random(c["salt"])
    got = [(c["new"], c["ctx"])]
    for _ in range(c["reqs"] - 1):
        n = c["new"] if c["new"] == 1 else rng.randint(max(1, c["new"] // 3), c["new"])
        cached = rng.randint((c["ctx"] - c["new"]) // 4, c["ctx"] - c["new"])
        if c["op"] in ("transfer", "restore") and c["reqs"] == 8:  # a batch of whole requests
            cached = c["ctx"] - n
        got.append((n, n + cached))
    return got


def _pairs(c):
    """Visible (query token, cached token) pairs of one head, and cached tokens that some query sees."""
    pairs = seen = 0
    for n, t in _lengths(c):
        w = c["window"] or t
        last = [t - n + i + 1 if c["causal"] else t for i in range(n)]
        pairs += sum(min(w, x) for x in last)
        seen += max(last) - max(0, min(last) - w)
    return pairs, seen


def work(case):
    c = case
    lens = _lengths(c)
    T = sum(n for n, _ in lens)
    row, row4 = c["dim"] * 2, c["dim"] // 2 + c["dim"] // 32
    if c["op"] == "append":
        # the rows of q, k and v, the rotated q, what the cache's rows stand for, and those rows themselves
        return {"bytes": T * ((2 * c["heads"] + 4 * c["kv_heads"]) * row + 2 * c["kv_heads"] * row4) + T * 8 * (c["axes"] + 1),
                "flops": T * (c["heads"] + c["kv_heads"]) * c["rot"] * 3 + T * 2 * c["kv_heads"] * c["dim"] * 4}
    if c["op"] == "attend":
        pairs, seen = _pairs(c)
        table = 4 * sum(-(-t // c["block"]) for _, t in lens)
        return {"bytes": 2 * T * c["heads"] * row + 4 * T * c["heads"] + 2 * seen * c["kv_heads"] * row4 + table,
                "flops": 4 * c["dim"] * pairs * c["heads"]}
    rows = c["layers"] * sum(-(-t // c["block"]) for _, t in lens) * c["block"] * 2 * c["kv_heads"]
    times = 2 if c["op"] == "transfer" else 1
    return {"bytes": times * rows * (row + row4), "flops": times * rows * c["dim"] * 4}


# ----------------------------------------------------------------------------------------
# the 4-bit format
# ----------------------------------------------------------------------------------------

def _plane_bytes(block, dim):
    """Bytes of one head's K or V of a block: elements, then scales, filled up to 16."""
    return (block * (dim // 2 + dim // 32) + 15) // 16 * 16


def _exponents(top, most):
    """Exponents of the scales of groups whose largest magnitudes these are."""
    m, e = torch.frexp(top)  # top = m 2^e, 0.5 <= m < 1
    e = e - 3 + (m >= 0.875).int()
    return torch.where(top > 0, e, -127).clamp(-127, most)


def _codes(y):
    """Codes of scaled elements: the nearest value, of two the one with the even code."""
    a = y.abs()
    c = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
    return c + torch.signbit(y).to(torch.uint8) * 8


def _values(codes):
    """What codes (0 to 15) stand for, before the scale."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    return table[codes.int()]


def _powers(scales):
    """2^(s - 127) of scale bytes, in 32 bits."""
    s = scales.int()
    return torch.where(s == 0, 1 << 22, s << 23).view(torch.float32)


def _groups(x, most):
    """(codes [..., groups, 32], scale bytes [..., groups]) of rows [..., dim]."""
    g = x.unflatten(-1, (-1, 32))
    e = _exponents(g.abs().amax(-1), most)
    # two factors: one alone may lie outside the numbers
    half = torch.div(-e, 2, rounding_mode="floor")
    y = g * torch.ldexp(torch.ones_like(half, dtype=g.dtype), half)[..., None]
    return _codes(y * torch.ldexp(torch.ones_like(half, dtype=g.dtype), -e - half)[..., None]), (e + 127).to(torch.uint8)


def _held(x, most):
    """Rows as the cache holds them, in 32 bits."""
    codes, scales = _groups(x, most)
    return (_values(codes) * _powers(scales)[..., None]).flatten(-2)


def _as_planes(cache, layout):
    """A 4-bit cache as [blocks][heads][K, V][plane], whatever its layout."""
    return cache if layout == 0 else cache.transpose(1, 2) if layout == 1 else cache.permute(1, 2, 0, 3)


def _rows_of(planes, block, dim):
    """Planes [..., plane] as rows in 32 bits: [..., block][dim]."""
    table = _values(torch.stack([torch.arange(256, device=planes.device) % 16, torch.arange(256, device=planes.device) // 16], 1))
    n = block * dim // 2
    x = table[planes[..., :n].int()].flatten(-2).unflatten(-1, (block, dim // 32, 32))
    scales = planes[..., n:n + block * (dim // 32)].unflatten(-1, (block, dim // 32))
    return (x * _powers(scales)[..., None]).flatten(-2)


def _new_planes(gen, dev, count, block, dim, gain, most):
    """`count` planes of random rows, elements of channel i times gain[i]."""
    out = torch.zeros(count, _plane_bytes(block, dim), dtype=torch.uint8, device=dev)
    n = block * dim // 2
    for a in range(0, count, 1 << 15):
        b = min(count, a + (1 << 15))
        codes, scales = _groups(torch.randn(b - a, block, dim, generator=gen, device=dev) * gain, most)
        codes = codes.flatten(1)
        out[a:b, :n] = codes[:, 0::2] | codes[:, 1::2] << 4
        out[a:b, n:n + block * (dim // 32)] = scales.flatten(1)
    return out


# ----------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------

def _as_tokens(cache, layout):
    """A 16-bit cache (or layers of them) as [...blocks][tokens of a block][K, V][heads][dim], whatever its layout."""
    if layout == 1:
        return cache.transpose(-4, -3)
    if layout == 2:
        return cache.movedim(-5, -3)
    return cache


def _ids(rng, counts, room, run):
    """Block ids of every request: runs of neighbours, about `run` long, in a shuffled pool."""
    cuts, at = [], 0
    while at < room:
        n = min(room - at, rng.randint(max(1, run // 2), run + run // 2))
        cuts.append(range(at, at + n))
        at += n
    rng.shuffle(cuts)
    flat = [i for c in cuts for i in c]
    return [flat[sum(counts[:r]):sum(counts[:r + 1])] for r in range(len(counts))]


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dt, most = DTYPES[c["dtype"]], MOST[c["dtype"]]
    lens = _lengths(c)
    R, H, Hk, D, bs = c["reqs"], c["heads"], c["kv_heads"], c["dim"], c["block"]
    new, ctx = [n for n, _ in lens], [t for _, t in lens]
    T = sum(new)
    counts = [-(-t // bs) for t in ctx]
    s = {"case": dict(c)}

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=dt)

    # a few channels of K are several times larger than the others
    gain = torch.where(torch.rand(D, generator=gen, device=dev) < 0.06, 4.0, 1.0)
    if c["op"] in ("transfer", "restore"):
        L, N, rng = c["layers"], sum(counts), random.Random(int(seed))
        room = N + N // 16 + 3

        def layers():
            return {0: (L, room, bs, 2, Hk, D), 1: (L, room, 2, bs, Hk, D), 2: (L, 2, room, bs, Hk, D)}[c["layout"]]

        offsets = [sum(counts[:r]) for r in range(R + 1)]
        s.update(offsets=torch.tensor(offsets, dtype=torch.int64, device=dev), total=N, room=room)
        s["dst"] = torch.zeros(layers(), dtype=dt, device=dev)
        s["dst_bases"] = torch.tensor([s["dst"][i].data_ptr() for i in range(L)], dtype=torch.int64, device=dev)
        s["dst_ids"] = torch.tensor(sum(_ids(rng, counts, room, c["run"] if c["op"] == "restore" else 1), []), dtype=torch.int32, device=dev)
        s["dst_runs"] = torch.zeros(N, 4, dtype=torch.int64, device=dev), torch.zeros(1, dtype=torch.int64, device=dev)
        if c["op"] == "transfer":
            s["src"] = randn(*layers())
            s["src"] *= gain.to(dt)
            s["src_bases"] = torch.tensor([s["src"][i].data_ptr() for i in range(L)], dtype=torch.int64, device=dev)
            s["src_ids"] = torch.tensor(sum(_ids(rng, counts, room, c["run"]), []), dtype=torch.int32, device=dev)
            s["src_runs"] = torch.zeros(N, 4, dtype=torch.int64, device=dev), torch.zeros(1, dtype=torch.int64, device=dev)
            s["buffer"] = torch.zeros(L * N, Hk, 2, _plane_bytes(bs, D), dtype=torch.uint8, device=dev)
        else:
            s["buffer"] = _new_planes(gen, dev, L * N * Hk * 2, bs, D, gain, most).view(L * N, Hk, 2, -1)
        return s

    # as many blocks as the batch holds; the rows that a call appends go to slots of a few of them
    blocks = sum(counts) if c["op"] == "attend" else -(-T // bs)
    room = blocks + 7
    shape = {0: (room, Hk, 2), 1: (room, 2, Hk), 2: (2, room, Hk)}[c["layout"]]
    planes = _new_planes(gen, dev, room * Hk * 2, bs, D, gain, most).view(room, Hk, 2, -1)
    s["cache"] = torch.empty(*shape, planes.shape[-1], dtype=torch.uint8, device=dev)
    _as_planes(s["cache"], c["layout"]).copy_(planes)
    del planes
    s.update(lens=torch.tensor(ctx, dtype=torch.int64, device=dev),
             offsets=torch.tensor([sum(new[:r]) for r in range(R + 1)], dtype=torch.int64, device=dev), T=T,
             max_new=max(new), max_ctx=max(ctx),
             tok_req=torch.tensor([r for r in range(R) for _ in range(new[r])], dtype=torch.int64, device=dev),
             tok_i=torch.tensor([i for r in range(R) for i in range(new[r])], dtype=torch.int64, device=dev))
    if c["op"] == "append":
        half = c["rot"] // 2
        s.update(q=randn(T, H, D), k=randn(T, Hk, D) * gain.to(dt), v=randn(T, Hk, D), q_out=torch.empty(T, H, D, dtype=dt, device=dev),
                 k_out=torch.empty(T, Hk, D, dtype=dt, device=dev), v_out=torch.empty(T, Hk, D, dtype=dt, device=dev))
        order = torch.randperm(room, generator=gen, device=dev)
        i = torch.arange(T, device=dev)
        s["slots"] = order[i // bs] * bs + i % bs
        place = (s["lens"] - s["offsets"].diff())[s["tok_req"]] + s["tok_i"]  # the token's place in its request
        # time, height and width of a grid of patches; one axis: the place itself
        axes = [place, place // 24 % 18, place % 24, place // 432]
        s["positions"] = torch.stack(axes[:c["axes"]])
        s["inv_freq"] = (1e6 ** (-torch.arange(half, dtype=torch.float64) / half)).to(torch.float32).to(dev)
        cut = [half * (a + 1) // c["axes"] for a in range(c["axes"])]
        s["pair_axis"] = [next(a for a, x in enumerate(cut) if i < x) for i in range(half)]
        s["pair_axis_dev"] = torch.tensor(s["pair_axis"], dtype=torch.int64, device=dev)
    else:
        width = max(counts)
        ids = torch.randperm(room, generator=gen, device=dev).to(torch.int32)
        s["table"] = torch.full((R, width), -1, dtype=torch.int32, device=dev)
        for r, n in enumerate(counts):
            s["table"][r, :n] = ids[sum(counts[:r]):sum(counts[:r]) + n]
        s["q"] = randn(T, H, D) * 1.5
        s["scale"] = D ** -0.5
        s["out"] = torch.empty(T, H, D, dtype=dt, device=dev)
        s["lse"] = torch.empty(T, H, dtype=torch.float32, device=dev)
    return s


# ----------------------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------------------

def _gathered(s, which):
    """K (0) or V (1) of every request's context in 32 bits: [reqs][kv_heads][max context][dim]."""
    c = s["case"]
    planes = _as_planes(s["cache"], c["layout"])[:, :, which][s["table"].clamp(min=0).long()]  # [reqs][blocks][heads][plane]
    return _rows_of(planes, c["block"], c["dim"]).transpose(1, 2).flatten(2, 3)[:, :, :s["max_ctx"]]


def _scores(s):
    """Scaled scores with -inf where a query does not see a slot: [reqs][kv_heads][new tokens x group][max context]."""
    c = s["case"]
    R, N, M, Hk, D = c["reqs"], s["max_new"], s["max_ctx"], c["kv_heads"], c["dim"]
    G = c["heads"] // Hk
    at = (s["offsets"][:-1, None] + torch.arange(N, device=s["q"].device)).clamp(max=s["T"] - 1)
    q = s["q"].float()[at].view(R, N, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(R, Hk, N * G, D)
    k = _gathered(s, 0).transpose(2, 3).contiguous()
    scores = torch.matmul(q, k).mul_(s["scale"])
    i, j = torch.arange(N, device=q.device)[None, :, None], torch.arange(M, device=q.device)[None, None, :]
    n, t = s["offsets"].diff()[:, None, None], s["lens"][:, None, None]
    last = t - n + i
    hidden = (j > last) if c["causal"] else (j >= t)
    if c["window"]:
        hidden = hidden | (j <= (last if c["causal"] else t - 1) - c["window"])
    hidden = hidden | (i >= n)
    return scores.view(R, Hk, N, G, M).masked_fill_(hidden[:, None, :, None, :], -math.inf).view(R, Hk, N * G, M)


def _from_padded(s, x):
    """[reqs][kv_heads][new tokens x group]... -> [tokens][heads]..."""
    c = s["case"]
    G = c["heads"] // c["kv_heads"]
    x = x.reshape(c["reqs"], c["kv_heads"], s["max_new"], G, *x.shape[3:])
    x = x.transpose(1, 2)[s["tok_req"], s["tok_i"]]
    return x.reshape(s["T"], c["heads"], *x.shape[3:])


def _plain_attend(s):
    p = _scores(s)
    top = p.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    p = p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, _gathered(s, 1).contiguous()) / torch.where(total > 0, total, 1.0)
    return [_from_padded(s, o).to(s["out"].dtype), _from_padded(s, (total.log() + top).squeeze(-1))]


def _plain_append(s):
    c = s["case"]
    half, bs, D, most = c["rot"] // 2, c["block"], c["dim"], MOST[c["dtype"]]
    angle = s["positions"][s["pair_axis_dev"]].t().double() * s["inv_freq"].double()

    def turned(x, of):
        y, cos, sin = x.to(of), angle.cos().to(of)[:, None], angle.sin().to(of)[:, None]
        if c["interleaved"]:
            a, b = y[..., 0:c["rot"]:2], y[..., 1:c["rot"]:2]
            z = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = y[..., :half], y[..., half:c["rot"]]
            z = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([z, y[..., c["rot"]:]], -1)

    # K in 64 bits up to its code: some elements lie next to a border between two of them
    planes = _as_planes(s["cache"], c["layout"])
    block, row, n = s["slots"] // bs, s["slots"] % bs, bs * D // 2
    i, j = torch.arange(D // 2, device=row.device), torch.arange(D // 32, device=row.device)
    kv = torch.stack([turned(s["k"], torch.float64), s["v"].double()], 2)  # [tokens][heads][K, V][dim]
    codes, scales = _groups(kv, most)
    held = (_values(codes) * _powers(scales)[..., None]).flatten(-2).to(s["k"].dtype)
    codes = codes.flatten(-2)
    planes[block[:, None], :, :, row[:, None] * (D // 2) + i] = (codes[..., 0::2] | codes[..., 1::2] << 4).permute(0, 3, 1, 2)
    planes[block[:, None], :, :, n + row[:, None] * (D // 32) + j] = scales.permute(0, 3, 1, 2)
    return [turned(s["q"], torch.float32).to(s["q"].dtype), held[:, :, 0], held[:, :, 1]]


def _plain_transfer(s):
    c = s["case"]
    x = _as_tokens(s["src"], c["layout"])[:, s["src_ids"].long()].float()
    _as_tokens(s["dst"], c["layout"])[:, s["dst_ids"].long()] = _held(x, MOST[c["dtype"]]).to(s["dst"].dtype)
    return s["dst"]


def _plain_restore(s):
    c = s["case"]
    rows = _rows_of(s["buffer"], c["block"], c["dim"]).to(s["dst"].dtype)  # [layers x blocks][heads][K, V][tokens][dim]
    _as_tokens(s["dst"], c["layout"])[:, s["dst_ids"].long()] = rows.permute(0, 3, 2, 1, 4).unflatten(0, (c["layers"], -1))
    return s["dst"]


# ----------------------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------------------

def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return {"append": _plain_append, "attend": _plain_attend, "transfer": _plain_transfer, "restore": _plain_restore}[op](s)
    from block_table_contiguous_amd import kvx as K

    if op == "append":
        K.kvx_rope_and_cache_fp4(s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["pair_axis"], s["slots"], s["cache"],
                                 s["q_out"], s["k_out"], s["v_out"], layout=LAYOUTS4[c["layout"]], interleaved=c["interleaved"])
        return [s["q_out"], s["k_out"], s["v_out"]]
    if op == "attend":
        bounds = dict(max_query_len=s["max_new"], max_context_len=s["max_ctx"], layout=LAYOUTS4[c["layout"]])
        if "workspace" not in s:  # kept with the batch, as a serving loop keeps it
            s["workspace"] = K.new_attention_workspace_fp4(s["q"], s["cache"], c["reqs"], s["max_new"], s["max_ctx"],
                                                           layout=LAYOUTS4[c["layout"]])
        K.kvx_paged_attention_fp4(s["q"], s["cache"], s["table"], s["offsets"], s["lens"], s["out"], s["lse"], scale=s["scale"],
                                  causal=c["causal"], window=c["window"], workspace=s["workspace"], **bounds)
        return [s["out"], s["lse"]]
    if op == "transfer":
        K.kvx_build_xfer_list(s["src_ids"], None, s["offsets"], K.MODE_PACK, *s["src_runs"])
        K.kvx_pack_fp4(s["src_bases"], s["src"][0], *s["src_runs"], s["total"], s["buffer"], layout=LAYOUTS[c["layout"]])
    K.kvx_build_xfer_list(None, s["dst_ids"], s["offsets"], K.MODE_UNPACK, *s["dst_runs"])
    K.kvx_unpack_fp4(s["buffer"], s["dst_bases"], s["dst"][0], *s["dst_runs"], s["total"], layout=LAYOUTS[c["layout"]])
    return s["dst"]


# ----------------------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------------------

def _exact_held(x, most):
    """Rows in 64 bits -> what the cache would hold: every group's nearest values by their distances."""
    g = x.reshape(*x.shape[:-1], -1, 32)
    top = g.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.floor(torch.log2(top / 7)) + 1, -127.0).clamp(-127, most)
    step = torch.pow(2.0, e)
    y, best, at = (g / step).abs(), torch.full_like(g, math.inf), torch.zeros_like(g)
    for value in (0.0, 1.0, 2.0, 4.0, 0.5, 1.5, 3.0, 6.0):  # even codes first: of two as near the first stays
        d = (y - value).abs()
        at, best = torch.where(d < best, value, at), torch.minimum(d, best)
    return (at * step * torch.sign(g)).reshape(x.shape)


def _exact_rows(plane, block, dim):
    """A plane's rows in 64 bits, from its bytes: sign, two bits of exponent, one of fraction."""
    n = block * dim // 2
    b = plane[..., :n].long()
    code = torch.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], block, dim // 32, 32)
    exp, frac = (code >> 1 & 3).double(), (code & 1).double()
    mag = torch.where(exp > 0, torch.pow(2.0, exp - 1) * (1 + frac / 2), frac / 2)
    s = plane[..., n:n + block * dim // 32].double().reshape(*b.shape[:-1], block, dim // 32, 1)
    return (torch.where(code >= 8, -mag, mag) * torch.pow(2.0, s - 127)).reshape(*b.shape[:-1], block, dim)


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    lens, H, Hk, D, bs = _lengths(c), c["heads"], c["kv_heads"], c["dim"], c["block"]
    if c["op"] in ("transfer", "restore"):
        dst = s["dst"].double()
        for l in range(c["layers"]):
            to = _as_tokens(dst[l], c["layout"])
            if c["op"] == "transfer":
                to[s["dst_ids"].long()] = _exact_held(_as_tokens(s["src"][l], c["layout"])[s["src_ids"].long()].double(), MOST[c["dtype"]])
            else:
                planes = s["buffer"][l * s["total"]:(l + 1) * s["total"]]
                to[s["dst_ids"].long()] = _exact_rows(planes, bs, D).permute(0, 3, 2, 1, 4)
        return dst
    if c["op"] == "append":
        half = c["rot"] // 2
        axis = s["positions"].double()[s["pair_axis_dev"]]
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=axis.device), (axis * s["inv_freq"].double()[:, None]).t())

        def turned(x):
            y = x.double().clone()
            first = slice(0, c["rot"], 2) if c["interleaved"] else slice(0, half)
            second = slice(1, c["rot"], 2) if c["interleaved"] else slice(half, c["rot"])
            z = torch.complex(y[..., first], y[..., second]) * turn[:, None, :]
            y[..., first], y[..., second] = z.real, z.imag
            return y

        return [turned(s["q"]), _exact_held(turned(s["k"]), MOST[c["dtype"]]), _exact_held(s["v"].double(), MOST[c["dtype"]])]
    planes = _as_planes(s["cache"], c["layout"])
    out = torch.zeros(s["T"], H, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["T"], H, dtype=torch.float64, device="cuda")
    at = 0
    for r, (n, t) in enumerate(lens):
        blocks = s["table"][r].long()[:-(-t // bs)]
        first = torch.arange(n, device="cuda")
        last = t - n + first if c["causal"] else torch.full((n,), t - 1, device="cuda")
        j = torch.arange(t, device="cuda")
        seen = (j <= last[:, None]) & ((j > last[:, None] - c["window"]) if c["window"] else (j >= 0))
        for g in range(Hk):
            kv = [_exact_rows(planes[blocks, g, w], bs, D).reshape(-1, D)[:t] for w in (0, 1)]
            for h in range(g * (H // Hk), (g + 1) * (H // Hk)):
                x = s["q"][at:at + n, h].double() @ kv[0].t() * s["scale"]
                x = torch.where(seen, x, -math.inf)
                lse[at:at + n, h] = torch.logsumexp(x, 1)
                out[at:at + n, h] = torch.softmax(x, 1) @ kv[1]
        at += n
    return [out, lse]
