"""Chunk attention with windows that leave nothing out, with and without rows before the first token (GPU).

Tolerances are test_chunk_attention's.
"""

import time

import pytest
import torch

from bucketized_guidance_step_gb300 import decode
from tests.test_chunk_attention import check, queries, run
from tests.test_decode_attention import BF16, F16, F32, build

pytestmark = pytest.mark.gpu

MOST = 2 ** 31 - 1


@pytest.mark.parametrize("dtype,dim", [(BF16, 64), (F16, 192), (F32, 32)])
@pytest.mark.parametrize("window,sinks", [(MOST, 0), (MOST, MOST), (MOST - 1, 3), (2 ** 30 + 1, MOST), (1, MOST), (40, MOST)])
def test_rows_before_the_first_token(dtype, dim, window, sinks):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = build([5, 0, 40, 150, 2], dim=dim, dtype=dtype, seed=3, status=status)
    seq, new = [0, 1, 2, 3, 4], [300, 9, 43, 150, 700]
    q = queries(cache, sum(new), 2)
    run(cache, q, seq, new)                             # (loads the kernel)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    out, lse = run(cache, q, seq, new, window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 0.15              # (no wait has run out: they last 0.2 s)
    assert int(status) == decode.GS_DEV_BAD_SEQ
    check(cache, 1, q, out, lse, seq, new, window=window, sinks=sinks)
    plain = run(cache, q, seq, new)                     # all that a row sees without a window
    assert torch.equal(out, plain[0]) and torch.equal(lse, plain[1])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_windows_past_every_position(dtype):
    cache = build([700, 130, 1], dtype=dtype, seed=1)
    seq, new = [0, 1, 2], [70, 130, 1]
    q = queries(cache, sum(new), 2)
    want = run(cache, q, seq, new)
    for window, sinks in ((MOST, 0), (2 ** 30, 0), (MOST, MOST)):
        got = run(cache, q, seq, new, window=window, sinks=sinks)
        check(cache, 1, q, *got, seq, new, window=window, sinks=sinks, rows=[[0, 69], [0, 64, 129], [0]])
