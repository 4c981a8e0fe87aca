"""The expert product where a resource is shortest, an expert of one row at every kernel and
number of K blocks, and with a capacity far above the rows (one rank's share of the experts).
The bound is test_gpu_block_gemm's."""
from __future__ import annotations

import pytest

from test_gpu_block_gemm import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [16, 112, 128, 144, 400])
@pytest.mark.parametrize("counts,N,slack", [
    ([1], 1032, 0), ([1, 1, 1], 2040, 0),         # waves that share K
    ([1] * 9, 4104, 0),                           # 32 x 128, one workgroup per CU
    ([1] * 40, 1032, 0),                          # 32 x 128, several
    ([100, 1, 1], 4104, 5),                       # 128 x 128
    ([1] * 5, 12296, 100),
    ([1, 383, 1], 16400, 200),                    # 256 x 256
])
def test_experts_of_one_row(counts, N, K, slack):
    check(counts, N, K, slack=slack, seed=K + N)


@pytest.mark.parametrize("counts,N,K", [
    ([3, 0, 17, 40, 1, 9, 0, 5], 1032, 656), ([31] * 32, 512, 400), ([0, 200], 4104, 272), ([0, 0, 0, 0], 520, 128),
    ([5], 2048, 1040),
])
@pytest.mark.parametrize("times", [8, 40])
def test_capacity_far_above_the_rows(counts, N, K, times):
    """The kernel and its tiles go by the capacity; the rows past the last stay as they are."""
    check(counts, N, K, slack=(times - 1) * max(1, sum(counts)) + 7, seed=N + times)
