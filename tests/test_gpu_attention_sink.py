"""kvx_paged_attention where one slot takes nearly all the weight and the others still decide the result: an
attention sink whose V is zero in front of, behind or among a long tail of slots that weigh 2^-20 to 2^-30
each. What the tail gives must not get lost when its weights are rounded to the element type."""
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


def sink_case(seed, lens, at, far, dtype, dim=64, heads=2, kv_heads=1):
    """Slot `at` (of the cached ones, from the front or behind) of every request scores `far` above the others, which differ by
    a few tenths, and its V is zero; theirs is around 64."""
    case = A.Case(seed, lens, heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype)
    g = torch.Generator().manual_seed(seed + 1)
    case.q.zero_()
    case.q[:, :, 0], case.q[:, :, 1] = 1.0, 0.5
    rows = A.as_tokens(case.cache, case.layout)
    for r, (n, c) in enumerate(lens):
        b, o = case.where(r, range(c))
        rows[b, o, 0, :, 0] = 0
        rows[b, o, 0, :, 1] = (torch.randn((c, kv_heads), generator=g) * dim ** 0.5 * 0.5).to(case.dtype)
        rows[b, o, 1] = (64 + 8 * torch.randn((c, kv_heads, dim), generator=g)).to(case.dtype)
        b, o = case.where(r, [at if at >= 0 else c - n + at])
        rows[b, o, 0, :, 0] = far * dim ** 0.5
        rows[b, o, 0, :, 1] = 0
        rows[b, o, 1] = 0
    return case


def check(case, split, shared=None):
    """The results against 64 bits. attention()'s tolerance for fp16 counts 2^-25 of the largest weight for each slot,
    which is what this is about: a weight that is held 2^11 higher than the largest one's 1 has a smallest step of
    2^-24, so its rounding is off by 2^-25 there, 2^-36 of the largest weight, or by half a step of its own."""
    want, want_lse, tol, tol_lse = A.attention(case)
    if case.dtype == torch.float16:
        for r, (n, c) in enumerate(case.lens):
            at = slice(int(case.offsets[r]), int(case.offsets[r]) + n)
            big = case.rows_of(r)[0][:, 1].abs().amax((0, 2)).repeat_interleave(case.heads // case.kv_heads)  # by head
            tol[at] += c * (2.0 ** -36 - 2.0 ** -25) * big[:, None]
    assert bool((tol > 0).all()) and float((tol / want.abs()).max()) < 0.05  # what the tail gives is far above the tolerance
    dev = case.to()
    if shared is not None:
        n, c = max(n for n, _ in case.lens), max(c for _, c in case.lens)
        assert (kvx().attention_workspace_bytes(dev[0], dev[1], len(case.lens), n, c) > 0) == shared
    out, lse, bits = A.attend(case, dev, split=split)
    assert bits == 0
    A.check("out", out, want, tol)
    A.check("lse", lse, want_lse, tol_lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("far", [14.0, 18.0, 21.0])
@pytest.mark.parametrize("at", [0, 1500, -1], ids=["first", "middle", "last"])
@pytest.mark.parametrize("n", [1, 70], ids=["decode", "chunk"])
def test_tail_behind_a_sink(n, at, far, dtype):
    case = sink_case(50, [(n, 3001 + n), (n, 2100)], at, far, dtype)
    check(case, split=False)
    check(case, split=True, shared=True)


@pytest.mark.parametrize("dim", [40, 128, 256])
@pytest.mark.parametrize("n", [1, 70], ids=["decode", "chunk"])
def test_tail_behind_a_sink_at_other_dims(n, dim):
    case = sink_case(51, [(n, 2500)], 0, 18.0, "fp16", dim=dim, heads=4, kv_heads=2)
    check(case, split=False)
    check(case, split=True)


def test_long_tail():
    """A hundred thousand slots that weigh 2^-26 each: together 2^-9 of the sink."""
    check(sink_case(52, [(1, 100003)], 0, 18.0, "fp16"), split=True, shared=True)
