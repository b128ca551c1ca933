"""kvx_paged_attention with scores of millions to 10^12, as far as the element types reach: 32 bits then hold a score in steps of 1 to
65536, and the softmax is the slot with the largest one."""
import pytest
import torch

import attention_util as A
from gpu_util import log

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    log(f"start {request.node.name}")
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("split", [False, True], ids=["whole", "shared"])
@pytest.mark.parametrize("n", [1, 70], ids=["decode", "chunk"])
@pytest.mark.parametrize("dtype,q_scale,k_scale", [("fp16", 3e3, 1e2), ("fp16", 4e3, 1e3), ("fp16", 8e3, 8e3), ("bf16", 4e3, 1e3),
                                                   ("bf16", 1e5, 1e4), ("bf16", 1e7, 1e6)])
def test_scores_far_from_zero(dtype, q_scale, k_scale, n, split):
    case = A.Case(80, [(n, n + 900), (n, 2000)], heads=2, kv_heads=1, dim=64, dtype=dtype, q_scale=q_scale)
    rows = A.as_tokens(case.cache, case.layout)
    rows[:, :, 0] *= k_scale
    out, lse, bits = A.attend(case, case.to(), split=split)
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
