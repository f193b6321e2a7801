"""The rotation table's scaling by parts, pair by pair from its definition."""
import math

import numpy as np
import pytest

import block_scaled_precision_gemm_amd as bsg


@pytest.mark.parametrize("dim,base,f,n", [(64, 10000.0, 4.0, 4096), (128, 10000.0, 8.0, 2048), (32, 500000.0, 2.5, 8192)])
def test_pairs_between_the_ends_go_linearly_in_their_index(dim, base, f, n):
    half = dim // 2
    speed = [base ** (-i / half) for i in range(half)]
    # the (real) index of a pair that turns k times in n positions: n base^(-i / half) = 2 pi k
    ends = [half * math.log(n / (2 * math.pi * k)) / math.log(base) for k in (32, 1)]
    t = bsg.rope_table(2, dim, base=base, scaling=("parts", f, n))
    angle = np.arctan2(t[1, 1], t[1, 0])
    between = 0
    for i in range(half):
        slow = min(max((i - ends[0]) / (ends[1] - ends[0]), 0.0), 1.0)
        between += 0.0 < slow < 1.0
        assert angle[i] == pytest.approx(speed[i] * ((1 - slow) + slow / f), rel=1e-5)
    assert between >= 3
