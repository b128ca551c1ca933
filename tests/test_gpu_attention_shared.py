"""kvx_paged_attention where the batch's steps are shared out over the GPU and tiles are joined from parts: the masks, values and
tables that test_gpu_attention.py has for tiles that one workgroup computes whole. Every case makes sure that its
sizes are shared."""
import math

import numpy as np
import pytest
import torch

import attention_util as A
from gpu_util import kvx, log

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    log(f"start {request.node.name}")
    yield
    torch.cuda.synchronize()


def shared(case, causal=True, window=0, err=0, blind=False):
    """The call against 64 bits, with a workspace that the launch has to have; its out and lse. blind: every score is -inf,
    which leaves the 64-bit weights undefined and the result as for a row that sees nothing."""
    dev = case.to()
    n, c = max(n for n, _ in case.lens), max(int(c) for c in case.context)
    assert kvx().attention_workspace_bytes(dev[0], dev[1], len(case.lens), n, c) > 0, "these sizes are not shared out"
    out, lse, bits = A.attend(case, dev, causal, window)
    want, want_lse, tol, tol_lse = A.attention(case, causal, window)
    used = int(case.offsets[-1])
    assert bits == err
    A.check("lse", lse[:used], want_lse[:used], tol_lse[:used])
    if blind:
        assert bool((lse[:used] == -math.inf).all()) and bool((out[:used] == 0).all())
    else:
        A.check("out", out[:used], want[:used], tol[:used])
    assert bool((out[used:] == 7).all()) and bool((lse[used:] == 7).all()), "rows of nobody were written"
    return out, lse


def put(case, r, slot, which, d, x, head=0):
    b, o = case.where(r, [slot])
    A.as_tokens(case.cache, case.layout)[b, o, which, head, d] = x


# requests of one token, of a few, of more rows than 32 for the KV head, of more than 128
FORMS = {"decode": 1, "drafted": 5, "chunk": 20, "tiles": 70}


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("dtype,dim", [("bf16", 64), ("fp16", 128)])
def test_unseen_slots_may_hold_anything(form, dtype, dim):
    """NaN and infinities in K and V: the rows that see them get them, of V in their dimension alone, and no other row does;
    in the first part of a context, in a later one, and where the causal limit passes."""
    n = FORMS[form]
    c = n + 2500
    case = A.Case(70, [(n, c)], heads=4, kv_heads=1, dim=dim, dtype=dtype)
    if n > 1:  # the last token alone sees these, and the last two
        put(case, 0, c - 1, 1, 5, math.nan)
        put(case, 0, c - 2, 1, 17, math.inf)
        shared(case)
        put(case, 0, c - 1, 0, 3, math.nan)
        shared(case)
    case = A.Case(71, [(n, c)], heads=4, kv_heads=1, dim=dim, dtype=dtype)
    put(case, 0, 700, 1, 7, math.inf)   # every row sees these
    put(case, 0, 1900, 1, 9, -math.inf)
    put(case, 0, 30, 1, 33, math.nan)
    put(case, 0, 2000, 1, 33, math.inf)
    shared(case)
    put(case, 0, 1000, 0, 11, math.nan)  # and a score of NaN
    out, lse = shared(case)
    assert bool(out.isnan().all()) and bool(lse.isnan().all())
    shared(case, window=1100)  # slots up to 1400 and more are behind the window


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens", [[(3, 0), (5, 2), (1, 6000), (1, 0)], [(150, 70), (3, 0), (1, 6000), (40, 7)],
                                  [(1, 0), (30, 5000), (0, 0), (200, 20), (1, 1)]], ids=["drafted", "chunk", "behind"])
def test_rows_that_see_nothing(lens, causal):
    """More new tokens than context, and no context at all, beside a long request."""
    case = A.Case(72, lens, heads=4, kv_heads=1, dim=64, extra=3)
    out, lse = shared(case, causal)
    for r, (n, c) in enumerate(lens):
        at = int(case.offsets[r])
        blind = n if c == 0 else max(0, n - c) if causal else 0
        assert bool((out[at:at + blind] == 0).all()) and bool((lse[at:at + blind] == -math.inf).all())
    shared(case, causal, window=64)


@pytest.mark.parametrize("form", list(FORMS))
def test_infinite_scores(form):
    """Parts of a context whose scores are all -inf give nothing; where all parts are such the row counts as empty."""
    n = FORMS[form]
    c = n + 3000
    case = A.Case(73, [(n, c)], heads=4, kv_heads=1, dim=64)
    case.q[:, :, 0] = 1.0
    rows = A.as_tokens(case.cache, case.layout)
    for lo, hi in ((0, 900), (600, 2400), (0, c)):
        b, o = case.where(0, range(lo, hi))
        rows[b, o, 0, 0, 0] = -math.inf
        shared(case, blind=(lo, hi) == (0, c))
        b, o = case.where(0, range(lo, hi))
        rows[b, o, 0, 0, 0] = 0.25


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_maxima_far_apart(form, dtype):
    """Parts whose largest scores lie hundreds apart, in both orders: the lesser ones vanish, nothing overflows."""
    n = FORMS[form]
    c = n + 3000
    for up in (False, True):
        case = A.Case(74, [(n, c), (n, n + 1400)], heads=4, kv_heads=1, dim=64, dtype=dtype)
        rows = A.as_tokens(case.cache, case.layout)
        case.q[:, :, 0] = 8.0
        for r, (_, length) in enumerate(case.lens):
            b, o = case.where(r, range(length))
            ramp = torch.arange(length).float() / length * 400
            rows[b, o, 0, 0, 0] = (ramp if up else 400 - ramp).to(case.dtype)
        shared(case)
    shared(A.Case(75, [(n, c)], heads=4, kv_heads=1, dim=128, dtype=dtype, q_scale=200.0))


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("block", [16, 24])
def test_bad_tables(form, block):
    """Entries outside the cache in several shares of a context, a context past the table's row, and a negative one."""
    K = kvx()
    n = FORMS[form]
    case = A.Case(76, [(n, n + 4000), (n, n + 900)], heads=4, kv_heads=1, dim=64, block=block)
    last = (n + 4000 - 1) // block
    case.table[0, 3], case.table[0, 90], case.table[0, last], case.table[1, 0] = -1, case.num_blocks, 1 << 30, -(1 << 31)
    shared(case, err=K.DEVERR_BLOCK_RANGE)
    case = A.Case(77, [(n, n + 2000), (n, n + 64)], heads=4, kv_heads=1, dim=64, block=block)
    case.context[0] = 1 << 40
    case.table[1, case.table[1] < 0] = 0
    rows = A.as_tokens(case.cache, case.layout)
    rows[rows.isnan()] = 0.5
    shared(case, err=K.DEVERR_TABLE_RANGE)
    case = A.Case(78, [(n, n + 20), (n, n + 2064), (2, 50)], heads=4, kv_heads=1, dim=64, block=block)
    case.context[0] = -5
    shared(case, err=K.DEVERR_TABLE_RANGE)


def test_shares_of_many_requests_with_gaps():
    """More requests than a wavefront has lanes, some without tokens or context, a few long ones among them, and windows."""
    rng = np.random.default_rng(79)
    lens = [(int(n), int(c)) for n, c in zip(rng.integers(0, 3, 130), rng.choice([0, 1, 40, 300, 2500], 130, p=[.2, .2, .3, .25, .05]))]
    case = A.Case(79, lens, heads=3, kv_heads=1, dim=80, extra=2)
    shared(case)
    shared(case, causal=False)
    shared(case, window=100)
