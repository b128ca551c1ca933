"""Rotated keys below the smallest normal 32-bit number, written into a 4-bit cache: each has to be rounded from 64 bits to its
4-bit value at once. They stand a little beside the borders between two codes, by less than 32 bits can tell from the border itself."""
import numpy as np
import pytest
import torch

import fp4_util as F
from gpu_util import DEV, kvx, log
from test_gpu_rope import rotated

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    log(f"start {request.node.name}")
    yield
    torch.cuda.synchronize()


BORDERS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)
BLOCK, DIM, HALF = 16, 64, 32


def append(k, freq, interleaved):
    """k [tokens][1][64], all at position 1: checks the keys' bytes in the cache, and what key_out says they stand for."""
    K, T = kvx(), k.shape[0]
    pos, axis = torch.ones(1, T, dtype=torch.int64), [0] * HALF
    key = rotated(k, pos, freq, axis, interleaved)[0].numpy()  # exact but for 2^-52: see the callers
    codes, scales = F.quantise(key, F.MOST[k.dtype])
    cache = K.new_fp4_cache(-(-T // BLOCK), BLOCK, 1, DIM, DEV)
    ko, vo = torch.zeros_like(k, device=DEV), torch.zeros_like(k, device=DEV)
    K.kvx_rope_and_cache_fp4(None, k.to(DEV), torch.zeros_like(k, device=DEV), pos.to(DEV), freq.to(DEV), axis,
                             torch.arange(T, device=DEV), cache, None, ko, vo, interleaved=interleaved)
    torch.cuda.synchronize()
    got_codes, got_scales = F.from_planes(cache.cpu().numpy()[:, 0, 0], BLOCK, DIM)
    got_codes, got_scales = got_codes.reshape(-1, DIM)[:T], got_scales.reshape(-1, DIM // 32)[:T]
    assert np.array_equal(got_scales, scales[:, 0])
    wrong = got_codes != codes[:, 0]
    assert not wrong.any(), f"{int(wrong.sum())} of {wrong.size} codes, first key {key[:, 0][wrong][0].hex()}"
    assert torch.equal(ko.cpu(), torch.from_numpy(F.values(codes, scales)).to(k.dtype))
    return key


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("exponent", [-127, -126, -125])
def test_bf16_keys_beside_a_border(interleaved, exponent):
    """Both elements of a pair are b, the angle is 2^-30: they become b (1 - 2^-30) and b (1 + 2^-30), and with the angle's other
    sign the other way round. Their groups have the smallest exponents there are."""
    pairs = torch.tensor([s * b * 2.0 ** exponent for b in BORDERS for s in (1, -1)], dtype=torch.float64)
    k = torch.zeros(2, 1, DIM, dtype=torch.bfloat16)
    freq = torch.zeros(HALF)
    n = len(pairs)
    freq[:n] = 2.0 ** -30
    freq[n:2 * n] = -2.0 ** -30
    for i in range(2 * n):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + HALF)
        k[0, 0, a] = k[0, 0, b] = pairs[i % n]
        k[1, 0, a], k[1, 0, b] = pairs[i % n], -pairs[i % n]
    for i in (2 * n, HALF - 1):  # pairs without a turn
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + HALF)
        k[:, 0, a] = k[:, 0, b] = 6 * 2.0 ** exponent
    key = append(k, freq, interleaved)
    tiny = np.abs(key) < 2.0 ** -126
    assert (tiny & (key.astype(np.float32) != key)).sum() >= 16  # 32 bits do not hold them


@pytest.mark.parametrize("off", [2.0 ** -23, -(2.0 ** -24)])
def test_fp16_keys_beside_a_border(off):
    """fp16 keys are no smaller than 2^-24, so a turned one is that small where its own element is 0: m 2^-24 times the sine of an
    angle of 2^-105 (1 + off). The pair's other element stays normal, in a group of its own, as the pairs stand half apart."""
    k = torch.zeros(2, 1, DIM, dtype=torch.float16)
    freq = torch.full((HALF,), 2.0 ** -105 * (1 + off))
    for i in range(HALF):
        k[0, 0, i] = 4 * BORDERS[i % 7] * 2.0 ** -24  # key i + 32 becomes border 2^-127 (1 + off)
        k[1, 0, i] = -4 * BORDERS[i % 7] * 2.0 ** -24 if i % 7 < 5 else 0
    key = append(k, freq, False)
    tiny = (key != 0) & (np.abs(key) < 2.0 ** -126)
    assert (tiny & (key.astype(np.float32) != key)).sum() >= 20


@pytest.mark.parametrize("interleaved", [False, True])
def test_bf16_keys_around_the_smallest_normal(interleaved):
    """Random keys from 2^-139 up to 2^-121, turned by any angle: subnormal and normal ones in one group."""
    g = torch.Generator().manual_seed(5)
    k = torch.randn(200, 1, DIM, generator=g) * 2.0 ** torch.randint(-15, -1, (200, 1, 1), generator=g)
    k = (k.double() * 2.0 ** -122).to(torch.bfloat16)
    freq = torch.rand(HALF, generator=g) * 6
    append(k, freq, interleaved)
