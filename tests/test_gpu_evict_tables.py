"""kvx_evict_compact with destination tables that hold the source's own blocks."""
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


def compact(case, dst, keep):
    K = kvx()
    cache, err = case.cache.to(DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    mass = torch.rand(*keep.shape[:2], 700, generator=torch.Generator().manual_seed(1))
    out = torch.full((*keep.shape[:2], keep.shape[2]), 5.0, device=DEV)
    K.kvx_evict_compact(cache, torch.from_numpy(case.table).to(DEV), dst.to(DEV), keep.to(DEV), mass.to(DEV), out,
                        layout=case.layout, err_flag=err)
    torch.cuda.synchronize()
    want = torch.where(keep >= 0, mass.gather(2, keep.long().clamp(min=0)), 0.0)
    assert torch.equal(out.cpu(), want)
    return cache.cpu(), int(err.item())


@pytest.mark.parametrize("cols", [44, 10], ids=["whole", "cut"])
@pytest.mark.parametrize("layout", A.LAYOUTS)
def test_a_copy_of_the_table_moves_nothing(cols, layout):
    """A copy of the source table, whole or cut to the columns that stay, is no move in place: the cache is left as it
    was and the bit is raised."""
    K = kvx()
    case = A.Case(60, [(1, 700), (1, 690)], heads=2, kv_heads=2, dim=64, layout=layout)
    keep = torch.arange(0, 600, 4, dtype=torch.int32)[:150].expand(2, 2, 150).contiguous()
    keep[0] += 3  # not even the first one stays
    got, bits = compact(case, torch.from_numpy(case.table[:, :cols].copy()), keep)
    assert bits == K.DEVERR_BLOCK_RANGE
    assert torch.equal(got.view(torch.int16), case.cache.view(torch.int16))


def test_rows_that_stay_in_a_copy_of_the_table():
    """Rows that are where they belong need no move, and raise nothing."""
    case = A.Case(61, [(1, 700)], heads=2, kv_heads=2, dim=128)
    keep = torch.arange(100, dtype=torch.int32).expand(1, 2, 100).contiguous()
    got, bits = compact(case, torch.from_numpy(case.table.copy()), keep)
    assert bits == 0
    assert torch.equal(got.view(torch.int16), case.cache.view(torch.int16))


@pytest.mark.parametrize("src_cols", [44, 3])
def test_a_kept_prefix_and_new_blocks_behind_it(src_cols):
    """The first blocks, kept whole, are the source's own; the rows behind them go to other blocks. The source table
    may be wider or narrower than the destination's."""
    case = A.Case(62, [(1, 700)], heads=2, kv_heads=2, dim=64, spare=60)
    case.table = np.ascontiguousarray(case.table[:, :src_cols])
    n = min(700, src_cols * 16)
    keep = torch.cat([torch.arange(32), torch.arange(33, n, 2), torch.full((n,), -1)])[:n].to(torch.int32).expand(1, 2, n).contiguous()
    free = np.setdiff1d(np.arange(case.num_blocks), case.table)
    dst = np.concatenate([case.table[0, :2], free])[None, :50].astype(np.int32)
    want = case.cache.clone()
    to, rows = A.as_tokens(want, case.layout), A.as_tokens(case.cache, case.layout)
    for i, k in enumerate(keep[0, 0].tolist()):
        if k >= 0:
            to[int(dst[0, i // 16]), i % 16] = rows[int(case.table[0, k // 16]), k % 16]
    got, bits = compact(case, torch.from_numpy(dst), keep)
    assert bits == 0
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
