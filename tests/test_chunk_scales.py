"""Chunk attention with the largest and smallest scales (GPU): scores of 0 stay 0.

Tolerances are test_chunk_attention's.
"""

import pytest
import torch

from tests.test_chunk_attention import check, queries, run
from tests.test_decode_attention import BF16, F16, F32, build

pytestmark = pytest.mark.gpu

MOST = torch.finfo(torch.float32).max


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("scale", [MOST, -MOST, 2.5e38, 1e-45, -1e-45])
@pytest.mark.parametrize("group", [2, 3])
def test_scores_of_zero(dtype, scale, group):
    cache = build([90, 300], dtype=dtype, seed=8)
    seq, new = [1, 0], [20, 90]
    q = queries(cache, sum(new), group)
    if abs(scale) > 1:
        q[:] = 0.0
    check(cache, 1, q, *run(cache, q, seq, new, scale=scale), seq, new, scale=scale)
