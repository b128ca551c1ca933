"""Cases, inputs, plain forms and 64-bit results of the operators that work on a paged KV cache:

  rope    rotary positions with one or several axes, and the write of the rotated rows through their slots
  attend  attention of each request's new tokens (one, or a chunk) over its paged cache
  mass    the attention weight that those tokens give to every cached token, added to a running total
  evict   the cached tokens with the most accumulated weight are kept and moved together

`run` computes a case in elementary torch operations, or with `own` set through the library's entry points.
Lengths follow from a case alone, the contents of the tensors from the seed.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
LAYOUTS = ("blocks_tokens_kv", "blocks_kv_tokens", "kv_blocks_tokens")


# ----------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------

def _case(op, name=None, **kw):
    c = {"op": op, "reqs": 1, "new": 1, "ctx": 1, "heads": 8, "kv_heads": 1, "dim": 128, "block": 16,
         "dtype": "bf16", "layout": LAYOUTS[0], "salt": 0}
    if op == "rope":
        c.update(axes=1, rot=128, interleaved=False)
    if op in ("attend", "mass"):
        c.update(causal=True, window=0)
    if op == "evict":
        c.update(budget=1, sink=4, recent=64)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one decode step of 8 requests on a one-KV-head shard: rotate 8 tokens and write them; latency counts
        _case("rope", "rope_decode", reqs=8, ctx=9216, salt=1),
        # a prefill of video tokens (time, height, width), 32 query and 8 KV heads
        _case("rope", "rope_video_prefill", reqs=4, new=4096, ctx=4096, heads=32, kv_heads=8, axes=3, salt=2),
        # the smallest decode: one request a few blocks long
        _case("attend", "attend_decode_small", ctx=129, salt=3),
        # a serving batch in decode: 32 requests of ragged lengths, 32 query and 8 KV heads
        _case("attend", "attend_decode_batch", reqs=32, ctx=8192, heads=32, kv_heads=8, salt=4),
        # decode of two long documents, K plane before V plane
        _case("attend", "attend_decode_long", reqs=2, ctx=131071, heads=32, kv_heads=8, dtype="fp16",
              layout=LAYOUTS[2], salt=5),
        # 8 requests of 576 blocks, each with a chunk of new tokens, one KV head (an 8-way head shard)
        _case("attend", "attend_chunk_shard", reqs=8, new=517, ctx=9216, salt=6),
        # the chunk of a long prompt: 2048 new tokens behind the cached ones
        _case("attend", "attend_chunk_long", new=2048, ctx=32768, heads=32, kv_heads=8, salt=7),
        # whole ragged prompts at a small head, 7 query heads a KV head, a sliding window
        _case("attend", "attend_prefill_window", reqs=5, new=1999, ctx=1999, heads=14, kv_heads=2, dim=64, dtype="fp16",
              layout=LAYOUTS[1], window=1024, salt=8),
        # after each decode step of a batch the step's weights are added to the totals
        _case("mass", "mass_decode_batch", reqs=32, ctx=8192, heads=32, kv_heads=8, salt=9),
        # the last 61 tokens of a long prompt vote on what the cache keeps
        _case("mass", "mass_last_tokens", reqs=2, new=61, ctx=32749, heads=32, kv_heads=8, salt=10),
        # one request's cache cut to its budget
        _case("evict", "evict_one", ctx=2100, kv_heads=1, budget=1024, salt=11),
        # a batch of 8 x 576 blocks cut to 4096 tokens a head
        _case("evict", "evict_batch", reqs=8, ctx=9216, kv_heads=8, budget=4096, salt=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "attend", "attend", "attend", "mass", "evict"])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 7, 8])
    dim = rng.choice([64, 64, 80, 128, 128, 128, 256])
    c = _case(op, reqs=_log_int(rng, 1, 48), heads=heads, kv_heads=kv_heads, dim=dim, block=rng.choice([16, 16, 16, 32, 64, 8, 24]),
              dtype=rng.choice(["bf16", "bf16", "fp16"]), layout=rng.choice(LAYOUTS), salt=rng.randrange(1 << 30))
    if op == "rope":
        c["new"] = _log_int(rng, 1, 4096)
        c["ctx"] = c["new"] + _log_int(rng, 1, 8192)
        c["axes"] = rng.choice([1, 2, 3, 4])
        c["rot"] = rng.choice([dim, dim, dim // 32 * 16])
        c["interleaved"] = rng.random() < 0.3
    elif op == "evict":
        c["ctx"] = _log_int(rng, 200, 32768)
        c["budget"] = max(100, int(c["ctx"] * rng.uniform(0.2, 0.9)))
        c["recent"] = rng.choice([0, 16, 64])
    else:
        long = 131072 if rng.random() < 0.3 else 16384
        c["new"] = rng.choice([1, 1, _log_int(rng, 2, 32 if op == "mass" else 2048), _log_int(rng, 2, 128)])
        c["ctx"] = c["new"] + _log_int(rng, 1, long)
        c["window"] = rng.choice([0, 0, 0, _log_int(rng, 16, 4096)])
        c["causal"] = rng.random() < 0.85
    most = {"rope": "rope_video_prefill", "attend": "attend_chunk_long", "mass": "mass_last_tokens", "evict": "evict_batch"}[op]
    top = work(next(x for x in listed() if x["name"] == most))
    # a drawn case costs no more than the largest of its kind, in work and in the plain form's scores
    while work(c)["bytes"] > max(top["bytes"], 1.1e9) or work(c)["flops"] > top["flops"] * (1 if op == "attend" else 4) or \
            c["reqs"] * c["heads"] * c["new"] * c["ctx"] > 2.2e9:
        if c["reqs"] > 1:
            c["reqs"] = (c["reqs"] + 1) // 2
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
    row = c["dim"] * 2
    if c["op"] == "rope":
        return {"bytes": T * (2 * c["heads"] + 4 * c["kv_heads"]) * row + T * 8 * (c["axes"] + 1),
                "flops": T * (c["heads"] + c["kv_heads"]) * c["rot"] * 3}
    if c["op"] == "evict":
        kept = sum(min(t, c["budget"]) for _, t in lens) * c["kv_heads"]
        return {"bytes": kept * (4 * row + 8) + 4 * c["kv_heads"] * sum(t for _, t in lens),
                "flops": c["kv_heads"] * sum(t for _, t in lens)}
    pairs, seen = _pairs(c)
    table = 4 * sum(-(-t // c["block"]) for _, t in lens)
    if c["op"] == "attend":
        return {"bytes": 2 * T * c["heads"] * row + 4 * T * c["heads"] + 2 * seen * c["kv_heads"] * row + table,
                "flops": 4 * c["dim"] * pairs * c["heads"]}
    return {"bytes": T * c["heads"] * (row + 4) + seen * c["kv_heads"] * (row + 8) + table,
            "flops": 2 * c["dim"] * pairs * c["heads"]}


# ----------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------

def _as_tokens(cache, layout):
    """The cache as [blocks][tokens of a block][K, V][heads][dim], whatever its layout."""
    if layout == LAYOUTS[1]:
        return cache.permute(0, 2, 1, 3, 4)
    if layout == LAYOUTS[2]:
        return cache.permute(1, 2, 0, 3, 4)
    return cache


def _tables(gen, dev, lens, block, room):
    """Block tables over a shuffled pool of `room` blocks, padded with -1, and the blocks not handed out."""
    counts = [-(-t // block) for t in lens]
    width = max(counts)
    ids = torch.randperm(room, generator=gen, device=dev).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=dev)
    at = 0
    for r, n in enumerate(counts):
        table[r, :n] = ids[at:at + n]
        at += n
    return table, ids[at:]


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dt = DTYPES[c["dtype"]]
    lens = _lengths(c)
    R, H, Hk, D, bs = c["reqs"], c["heads"], c["kv_heads"], c["dim"], c["block"]
    new, ctx = [n for n, _ in lens], [t for _, t in lens]
    T = sum(new)

    def randn(*shape, dtype=dt):
        return torch.randn(shape, generator=gen, device=dev, dtype=dtype)

    blocks = sum(-(-t // bs) for t in ctx)
    kept = [min(t, c["budget"]) for t in ctx] if c["op"] == "evict" else [0]
    room = blocks + sum(-(-t // bs) for t in kept) + 7
    table, free = _tables(gen, dev, ctx, bs, room)
    shape = {LAYOUTS[0]: (room, bs, 2, Hk, D), LAYOUTS[1]: (room, 2, bs, Hk, D), LAYOUTS[2]: (2, room, bs, Hk, D)}[c["layout"]]
    cache = randn(*shape)
    s = {"case": dict(c), "cache": cache, "table": table, "lens": torch.tensor(ctx, dtype=torch.int64, device=dev),
         "offsets": torch.tensor([sum(new[:r]) for r in range(R + 1)], dtype=torch.int64, device=dev), "T": T,
         "max_new": max(new), "max_ctx": max(ctx),
         "tok_req": torch.tensor([r for r in range(R) for _ in range(new[r])], dtype=torch.int64, device=dev),
         "tok_i": torch.tensor([i for r in range(R) for i in range(new[r])], dtype=torch.int64, device=dev)}
    if c["op"] == "rope":
        half = c["rot"] // 2
        s.update(q=randn(T, H, D), k=randn(T, Hk, D), v=randn(T, Hk, D), q_out=torch.empty(T, H, D, dtype=dt, device=dev))
        place = (s["lens"] - s["offsets"].diff())[s["tok_req"]] + s["tok_i"]  # the token's place in its request
        s["slots"] = table[s["tok_req"], place // bs].to(torch.int64) * bs + place % bs
        # time, height and width of a grid of patches; one axis: the place itself
        axes = [place, place // 24 % 18, place % 24, place // 432]
        s["positions"] = torch.stack(axes[:c["axes"]])
        s["inv_freq"] = (1e6 ** (-torch.arange(half, dtype=torch.float64) / half)).to(torch.float32).to(dev)
        cut = [half * (a + 1) // c["axes"] for a in range(c["axes"])]
        s["pair_axis"] = [next(a for a, x in enumerate(cut) if i < x) for i in range(half)]
        s["pair_axis_dev"] = torch.tensor(s["pair_axis"], dtype=torch.int64, device=dev)
    elif c["op"] == "evict":
        counts = [-(-t // bs) for t in kept]
        width = max(counts)
        dst = torch.full((R, width), -1, dtype=torch.int32, device=dev)
        for r, n in enumerate(counts):
            dst[r, :n] = free[sum(counts[:r]):sum(counts[:r]) + n]
        s["dst_table"] = dst
        wide = torch.arange(max(ctx), device=dev)[None, None, :] < s["lens"][:, None, None]
        # a few tokens gather most of the weight, and some get none at all
        w = torch.rand((R, Hk, max(ctx)), generator=gen, device=dev).pow_(8) * 50
        w = torch.where(torch.rand((R, Hk, max(ctx)), generator=gen, device=dev) < 0.05, 0.0, w)
        s["mass"] = torch.where(wide, w, 0.0)
        s["mass_out"] = torch.zeros((R, Hk, c["budget"]), device=dev)
        s["keep"] = torch.empty((R, Hk, c["budget"]), dtype=torch.int32, device=dev)
        s["new_lens"] = torch.empty(R, dtype=torch.int64, device=dev)
        s["max_kept"] = max(kept)
    else:
        s["q"] = randn(T, H, D) * 1.5
        s["scale"] = D ** -0.5
        s["out"] = torch.empty(T, H, D, dtype=dt, device=dev)
        s["lse"] = torch.empty(T, H, dtype=torch.float32, device=dev)
        if c["op"] == "mass":
            scores = _scores(s)
            s["lse"] = _from_padded(s, torch.logsumexp(scores, -1))
            s["mass"] = torch.rand((R, Hk, max(ctx)), generator=gen, device=dev) * (64 / max(ctx))  # some steps' totals
    return s


# ----------------------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------------------

def _gathered(s, which):
    """K (0) or V (1) of every request's context in 32 bits: [reqs][kv_heads][max context][dim]."""
    c = s["case"]
    j = torch.arange(s["max_ctx"], device=s["cache"].device)
    ids = s["table"][:, j // c["block"]].clamp(min=0).long()
    rows = _as_tokens(s["cache"], c["layout"])[:, :, which][ids, j % c["block"]]
    return rows.permute(0, 2, 1, 3).float()


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
    o = torch.matmul(p, _gathered(s, 1)) / torch.where(total > 0, total, 1.0)
    return [_from_padded(s, o).to(s["out"].dtype), _from_padded(s, (total.log() + top).squeeze(-1))]


def _plain_mass(s):
    c = s["case"]
    R, Hk, N, M = c["reqs"], c["kv_heads"], s["max_new"], s["max_ctx"]
    G = c["heads"] // Hk
    at = (s["offsets"][:-1, None] + torch.arange(N, device=s["q"].device)).clamp(max=s["T"] - 1)
    lse = s["lse"][at].view(R, N, Hk, G).transpose(1, 2).reshape(R, Hk, N * G, 1)
    p = _scores(s).sub_(lse).exp_()
    s["mass"] += p.double().sum(2).float() if N * G > 256 else p.sum(2)
    return s["mass"]


def _plain_rope(s):
    c = s["case"]
    half, bs = c["rot"] // 2, c["block"]
    angle = s["positions"][s["pair_axis_dev"]].t().double() * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x):
        y = x.float()
        if c["interleaved"]:
            a, b = y[..., 0:c["rot"]:2], y[..., 1:c["rot"]:2]
            z = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = y[..., :half], y[..., half:c["rot"]]
            z = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([z, y[..., c["rot"]:]], -1).to(x.dtype)

    _as_tokens(s["cache"], c["layout"])[s["slots"] // bs, s["slots"] % bs] = torch.stack([turned(s["k"]), s["v"]], 1)
    return [turned(s["q"]), s["cache"]]


def _plain_evict(s):
    c = s["case"]
    R, Hk, M, B, bs = c["reqs"], c["kv_heads"], s["max_ctx"], c["budget"], c["block"]
    dev = s["mass"].device
    j, t = torch.arange(M, device=dev), s["lens"][:, None, None]
    rank = torch.where((j < c["sink"]) | (j >= t - c["recent"]), math.inf, s["mass"])
    rank = torch.where(j < t, rank, -math.inf)
    if M < B:
        rank = torch.nn.functional.pad(rank, (0, B - M), value=-math.inf)
    best = rank.sort(dim=-1, descending=True, stable=True).indices[..., :B]
    new = s["lens"].clamp(max=B)
    there = torch.arange(B, device=dev) < new[:, None, None]
    best = torch.where(there, best, 1 << 40).sort(-1).values
    keep = torch.where(there, best, -1)
    # where a request keeps fewer rows than the longest one, its own source rows are written with what they hold
    n = s["max_kept"]
    from_ = keep[..., :n].clamp(min=0)
    src = s["table"].gather(1, (from_ // bs).view(R, -1)).view(R, Hk, n).long()
    i = torch.arange(n, device=dev)
    dst = s["dst_table"][:, i // bs].long()[:, None, :].expand(R, Hk, n)
    dst_off = (i % bs).expand(R, Hk, n)
    ok = (keep[..., :n] >= 0) & (dst >= 0)
    h = torch.arange(Hk, device=dev)[None, :, None].expand(R, Hk, n)
    view = _as_tokens(s["cache"], c["layout"])
    dst, dst_off = torch.where(ok, dst, src), torch.where(ok, dst_off, from_ % bs)
    for which in (0, 1):
        plane = view[:, :, which]
        plane[dst, dst_off, h] = plane[src, from_ % bs, h]
    s["mass_out"].copy_(torch.where(there, s["mass"].gather(2, keep.clamp(min=0, max=M - 1)), 0.0))
    return [keep.to(torch.int32), new, s["cache"], s["mass_out"]]


# ----------------------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------------------

def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return {"rope": _plain_rope, "attend": _plain_attend, "mass": _plain_mass, "evict": _plain_evict}[op](s)
    from block_table_contiguous_amd import kvx as K

    if op == "rope":
        K.kvx_rope_and_cache(s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["pair_axis"], s["slots"], s["cache"],
                             s["q_out"], layout=c["layout"], interleaved=c["interleaved"])
        return [s["q_out"], s["cache"]]
    if op == "evict":
        K.kvx_evict_select(s["mass"], s["lens"], c["budget"], c["sink"], c["recent"], s["keep"], s["new_lens"])
        K.kvx_evict_compact(s["cache"], s["table"], s["dst_table"], s["keep"], s["mass"], s["mass_out"],
                            layout=c["layout"])
        return [s["keep"], s["new_lens"], s["cache"], s["mass_out"]]
    bounds = dict(scale=s["scale"], causal=c["causal"], window=c["window"], max_query_len=s["max_new"],
                  max_context_len=s["max_ctx"], layout=c["layout"])
    if op == "attend":
        if "workspace" not in s:  # kept with the batch, as a serving loop keeps it
            s["workspace"] = K.new_attention_workspace(s["q"], s["cache"], c["reqs"], s["max_new"], s["max_ctx"],
                                                       layout=c["layout"])
        K.kvx_paged_attention(s["q"], s["cache"], s["table"], s["offsets"], s["lens"], s["out"], s["lse"],
                              workspace=s["workspace"], **bounds)
        return [s["out"], s["lse"]]
    K.kvx_attention_mass(s["q"], s["cache"], s["table"], s["offsets"], s["lens"], s["lse"], s["mass"], **bounds)
    return s["mass"]


# ----------------------------------------------------------------------------------------
# the definitions in 64 bits, request by request
# ----------------------------------------------------------------------------------------

def _rows(s, r, upto):
    """Request r's slots 0..upto-1 as (block, offset) index tensors."""
    j = torch.arange(upto, device=s["cache"].device)
    bs = s["case"]["block"]
    return s["table"][r].long()[torch.div(j, bs, rounding_mode="floor")], j % bs


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    lens, H, Hk, D = _lengths(c), c["heads"], c["kv_heads"], c["dim"]
    G = H // Hk
    tokens = _as_tokens(s["cache"], c["layout"])
    if c["op"] == "evict":
        cache, mass, bs = s["cache"].double(), s["mass"].cpu().numpy().astype("float64"), c["block"]
        total = torch.zeros(s["mass_out"].shape, dtype=torch.float64)
        for r, (_, t) in enumerate(lens):
            n = min(t, c["budget"])
            for h in range(Hk):
                value = mass[r, h, :t].copy()
                value[:c["sink"]] = value[max(0, t - c["recent"]):] = math.inf
                kept = sorted(sorted(range(t), key=lambda j: (-value[j], j))[:n])
                total[r, h, :n] = torch.from_numpy(mass[r, h, kept])
                j, i = torch.tensor(kept, device="cuda"), torch.arange(n, device="cuda")
                _as_tokens(cache, c["layout"])[s["dst_table"][r].long()[i // bs], i % bs, :, h] = \
                    tokens[s["table"][r].long()[j // bs], j % bs, :, h].double()
        return [None, None, cache, total]
    if c["op"] == "rope":
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

        cache = s["cache"].double()
        where = (s["slots"] // c["block"], s["slots"] % c["block"])
        _as_tokens(cache, c["layout"])[where[0], where[1], 0] = turned(s["k"])
        _as_tokens(cache, c["layout"])[where[0], where[1], 1] = s["v"].double()
        return [turned(s["q"]), cache]
    out = torch.zeros(s["T"], H, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["T"], H, dtype=torch.float64, device="cuda")
    mass = s["mass"].double() if c["op"] == "mass" else None
    at = 0
    for r, (n, t) in enumerate(lens):
        blk, off = _rows(s, r, t)
        kv = tokens[blk, off].double()
        first = torch.arange(n, device="cuda")
        last = t - n + first if c["causal"] else torch.full((n,), t - 1, device="cuda")
        j = torch.arange(t, device="cuda")
        seen = (j <= last[:, None]) & ((j > last[:, None] - c["window"]) if c["window"] else (j >= 0))
        for h in range(H):
            x = s["q"][at:at + n, h].double() @ kv[:, 0, h // G].t() * s["scale"]
            x = torch.where(seen, x, -math.inf)
            if c["op"] == "mass":
                mass[r, h // G, :t] += torch.exp(x - s["lse"][at:at + n, h, None].double()).sum(0)
                continue
            lse[at:at + n, h] = torch.logsumexp(x, 1)
            out[at:at + n, h] = torch.softmax(x, 1) @ kv[:, 1, h // G]
        at += n
    return mass if c["op"] == "mass" else [out, lse]
