"""kvx_paged_attention and kvx_attention_mass at the ends of what they count."""
import pytest
import torch

from gpu_util import DEV, kvx, log

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    log(f"start {request.node.name}")
    yield
    torch.cuda.synchronize()


def test_bad_offsets_with_more_tiles_than_32_bits():
    """Offsets that give the same 66000 tokens to 32768 requests: 2.16e9 tiles, past 2^31, for a workspace with slots for
    131535 and the shares. Nothing is written outside the tensors or the workspace, and the bit is raised."""
    K = kvx()
    T, R, heads, guard = 66000, 65535, 32, 1 << 16
    q = torch.zeros(T, heads, 8, dtype=torch.bfloat16, device=DEV)
    cache = torch.ones(4, 16, 2, 1, 8, dtype=torch.bfloat16, device=DEV)
    table = torch.zeros(R, 1, dtype=torch.int32, device=DEV)
    off = torch.zeros(R + 1, dtype=torch.int64, device=DEV)
    off[1::2] = T
    ctx = torch.full((R,), 16, dtype=torch.int64, device=DEV)
    out = torch.full((T + 2, heads, 8), 7.0, dtype=torch.bfloat16, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    n = K.attention_workspace_bytes(q, cache, R, 0, 1 << 20)
    assert n > 0  # the work is shared out, with parts in the workspace
    ws = torch.full((n + 2 * guard,), 0xA5, dtype=torch.uint8, device=DEV)
    K.kvx_paged_attention(q, cache, table, off, ctx, out[1:T + 1], workspace=ws[guard:guard + n], max_query_len=0,
                          max_context_len=1 << 20, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == K.DEVERR_OFFSETS
    assert bool((ws[:guard] == 0xA5).all()) and bool((ws[guard + n:] == 0xA5).all()), "written outside the workspace"
    assert bool((out[0] == 7).all()) and bool((out[T + 1] == 7).all())
