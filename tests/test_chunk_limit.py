"""How long chunk attention's waits may last (CPU): at least 0.2 s, and at least 7 times what a share takes.

A share of a 16-bit call has tiles of 256 rows (128 of heads over 128 dims), one of an fp32 call tiles of 64, with
costs in 16ths of a position and 288 positions beside a tile's own. RATES are measured times of one 16th.
"""

import os
import shutil
import subprocess

import pytest

from bucketized_guidance_step_gb300 import build

SOURCE = """
#include <cstdio>
#include <cstdlib>
#include "chunk_limit.h"
int main(int argc, char** argv) {
    for (int i = 1; i + 1 < argc; i += 2)
        printf("%llu\\n", gs_decode::chunk_limit_ns(atoll(argv[i]), argv[i + 1][0] == 'f' ? gs_decode::kChunkNsFp32 : gs_decode::kChunkNs));
    return 0;
}
"""

# type, rows of a tile, blocks, ns: heads of 128, 64 and 256; pages of one token (heads of 128 and 256) and of 33
RATES = [("h", 256, 152, 0.81), ("h", 256, 152, 0.79), ("h", 128, 152, 0.87), ("h", 256, 152, 6.44), ("h", 128, 152, 9.07),
         ("h", 256, 152, 2.32),
         # heads of 128, 64 and 256; scores of NaN (heads of 128 and 256)
         ("f", 64, 304, 14.1), ("f", 64, 304, 9.2), ("f", 64, 152, 15.8), ("f", 64, 304, 31.1), ("f", 64, 152, 37.0)]


@pytest.fixture(scope="module")
def limit():
    cc = shutil.which("g++") or shutil.which("c++")
    if cc is None:
        pytest.skip("no C++ compiler")
    folder = os.path.join(build.BUILD, "tests_tmp")
    os.makedirs(folder, exist_ok=True)
    src, exe = os.path.join(folder, "limit.cpp"), os.path.join(folder, "limit")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run([cc, "-std=c++17", "-I", build.CSRC_DECODE, src, "-o", exe], check=True)

    def of(cost, kind):
        return int(subprocess.run([exe, str(int(cost)), kind], check=True, capture_output=True, text=True).stdout)

    return of


def share(tokens, past, q_heads, kv_heads, rows, blocks):
    """A block's cost of one prompt of `tokens` behind `past`."""
    group = q_heads // kv_heads
    tiles = -(-tokens * group // rows)
    step = 16 * rows // group
    return kv_heads * (tiles * 16 * (288 + past) + step * tiles * (tiles + 1) // 2) // blocks


@pytest.mark.parametrize("tokens,past", [(1, 0), (2048, 14336), (180000, 0), (1 << 20, 0), (1 << 16, 1 << 24)])
def test_a_share_has_time(limit, tokens, past):
    for kind, rows, blocks, ns in RATES:
        cost = share(tokens, past, 32, 8, rows, blocks)
        got = limit(cost, kind)
        assert got >= 200_000_000 + 7 * cost * ns


def test_small_calls_wait_no_longer_than_before(limit):
    # 8 prompts of 2048 tokens: 0.2 s and a few per cent of it
    cost = 8 * share(2048, 0, 32, 8, 256, 152)
    assert 200_000_000 <= limit(cost, "h") <= 220_000_000


def test_no_cost_overflows(limit):
    for kind in "hf":
        before = 0
        for bits in range(0, 63):
            now = limit((1 << bits) - 1, kind)
            assert 200_000_000 <= now < 1 << 62 and now >= before
            before = now
