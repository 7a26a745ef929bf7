"""The linear unit at sizes that reach every tile height of the narrow kernel (32, 64 and 128 rows) with
every number of splits, ragged in each dimension, against float64 on the GPU. Bounds as in
test_linear_unit_wide."""
from __future__ import annotations

import pytest

from test_linear_unit_wide import check_dw, check_dx, check_forward, forward_case, z  # noqa: F401

pytestmark = pytest.mark.gpu

# (m, r, k, shards): the forward's tile rows x splits; dx's
SHAPES = [
    (31, 264, 136, 1),     # 32 x 1; 32 x 2
    (9, 1160, 264, 5),     # 32 x 2; 32 x 8
    (32, 520, 520, 5),     # 32 x 4; 32 x 4
    (2, 2056, 1032, 1),    # 32 x 8; 32 x 8
    (33, 136, 136, 1),     # 64 x 1; 64 x 1
    (64, 264, 328, 3),     # 64 x 2; 64 x 2
    (63, 776, 520, 1),     # 64 x 4; 64 x 4
    (65, 2056, 1160, 1),   # 64 x 4; 64 x 8
    (130, 1032, 2056, 3),  # 64 x 8; 64 x 4
    (700, 2312, 776, 1),   # 64 x 1; 64 x 2
    (100, 19592, 72, 1),   # 128 x 1; 64 x 8
    (127, 136, 19592, 1),  # 64 x 8; 128 x 1
    (1700, 776, 2312, 1),  # 128 x 2
    (1700, 2312, 776, 1),  # dx: 128 x 2
    (1150, 904, 5128, 1),  # 128 x 4
    (1150, 5128, 904, 1),  # dx: 128 x 4
    # copies of W cut to the shards' ends (shards of a multiple of 8 or 16 rows)
    (1700, 760, 2312, 5),  # 128 x 2
    (1700, 2280, 776, 5),  # dx: 128 x 2
    (2100, 1680, 520, 7),
    (300, 192, 392, 8),
    (5, 240, 1032, 6),
]


@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_forward(z, i):  # noqa: F811
    for j in (i, i + 7):
        check_forward(z, *SHAPES[i], *forward_case(j))


@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_dx(z, i):  # noqa: F811
    for j in (i, i + 7):
        act, _, has_res, bits8 = forward_case(j)
        check_dx(z, *SHAPES[i], act, has_res, bits8)


# 64 rows x 1, 2, 4, 8 splits; 128 x 2, 4; fp32: 128 x 8
@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("m,r,k", [(100, 264, 136), (300, 520, 776), (700, 264, 520), (1100, 136, 264),
                                   (3000, 1160, 904), (6100, 904, 776), (18700, 1160, 904)])
def test_dw(z, m, r, k, wide):  # noqa: F811
    check_dw(z, m, r, k, wide)
