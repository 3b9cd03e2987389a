"""Accumulated weights of more query rows than either kernel stages at once, and of as many as the first one
takes, against the fp64 oracle."""
from __future__ import annotations

import pytest
import torch

from tests.test_weights_evict_gpu import test_weights_match_oracle as check

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


@pytest.mark.parametrize("four,b,lens,H,G,paged,M,n_sel", [
    (False, 64, [900, 5], 1, 16, True, 20, 0),       # 320 rows, staged twice: the second pass adds to the first's sums
    (False, 128, [1300], 2, 9, False, 57, 5),        # 513 rows: three times, the last with one row
    (True, 128, [1300], 1, 9, True, 57, 0),
    (False, 64, [700, 64], 2, 9, True, 7, 0),        # 63 rows: the most of the register kernel's short launches
    (False, 64, [700, 64], 2, 16, True, 4, 0),       # 64: the least of the other's
    (True, 64, [700, 64], 2, 23 // 2, True, 2, 0),   # 22 rows of a four-bit cache: register kernel
    (False, 64, [40000, 300, 9000], 8, 11, True, 2, 0),   # 22 rows, long: equal shares, register kernel
    (False, 64, [40000, 300, 9000], 8, 12, True, 2, 0),   # 24 rows, long: tensor memory
])
def test_many_rows(four, b, lens, H, G, paged, M, n_sel):
    check(four, b, lens, H, G, paged, M, n_sel, False)
