"""The 4-bit format as the tests' own form has it, against hand-worked values (CPU)."""
import math

import numpy as np
import pytest

import fp4_util as F


def group(*first):
    x = np.zeros(32)
    x[:len(first)] = first
    return x


def test_values_and_ties():
    """With a 6 in the group its scale is 1: ties go to the even code."""
    x = group(6, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 2.6, 3.5, 5, 5.1, -0.25, -5.5, -1)
    codes, scales = F.quantise(x, 125)
    assert scales.tolist() == [127]
    assert codes[:14].tolist() == [7, 0, 1, 2, 2, 4, 4, 5, 6, 6, 7, 8, 15, 10]


@pytest.mark.parametrize("top,scale", [(6.99, 127), (7.0, 128), (8.0, 128), (13.9, 128), (14.0, 129), (1.0, 125), (0.875, 125),
                                       (0.8749, 124), (0.0, 0), (2.0 ** -140, 0), (2.0 ** 127 * 1.99, 252)])
def test_scales(top, scale):
    codes, scales = F.quantise(group(top), 125)
    assert scales.tolist() == [scale]
    v = F.values(codes, scales)
    if 2.0 ** -120 < top < 7 * 2.0 ** 125:
        assert abs(v[0] - top) <= 2.0 ** (scale - 127)  # half the spacing at the top


def test_fp16_stays_finite_and_bad_groups_are_nan():
    codes, scales = F.quantise(group(65504.0), 13)
    assert scales.tolist() == [140] and F.values(codes, scales)[0] == 49152
    for bad in (math.nan, math.inf, -math.inf):
        codes, scales = F.quantise(group(1, bad), 125)
        assert scales.tolist() == [255] and not codes.any() and np.isnan(F.values(codes, scales)).all()


@pytest.mark.parametrize("block,dim", [(1, 32), (16, 128), (24, 96), (3, 256)])
def test_planes_round_trip(block, dim):
    rng = np.random.default_rng(block)
    codes = rng.integers(0, 16, (2, block, dim)).astype(np.uint8)
    scales = rng.integers(0, 256, (2, block, dim // 32)).astype(np.uint8)
    planes = F.to_planes(codes, scales)
    assert planes.shape == (2, F.plane_bytes(block, dim)) and planes.shape[1] % 16 == 0
    assert planes[0, 0] == codes[0, 0, 0] | codes[0, 0, 1] << 4 and planes[1, block * dim // 2] == scales[1, 0, 0]
    c, s = F.from_planes(planes, block, dim)
    assert np.array_equal(c, codes) and np.array_equal(s, scales)
