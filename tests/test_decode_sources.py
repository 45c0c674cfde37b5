"""Rules of the decode kernels' sources that no run can show (CPU)."""

import os
import re

import pytest

from bucketized_guidance_step_gb300 import build


@pytest.mark.parametrize("name", ["guided_logits.cu", "paged_attention.cuh"])
def test_a_barrier_stands_between_the_count_of_parts_and_their_reading(name):
    """One thread counts the parts that have arrived; a shuffle of its answer orders no memory, so
    the other threads may read the parts only past a barrier that it takes part in."""
    with open(os.path.join(build.CSRC_DECODE, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    counts = [m.end() for m in re.finditer(r"atomicAdd\(p\.arrived", text)]
    assert len(counts) == 1
    between = text[counts[0]:text.index("__ldcg(", counts[0])]
    answer = max(between.rfind("__shfl_sync("), between.rfind("turn = last"))
    assert answer > 0 and re.search(r"__sync(warp|threads)\(\)", between[answer:])
