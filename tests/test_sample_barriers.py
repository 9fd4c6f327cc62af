"""Shared memory of the sampling kernel between barriers.  cta_exclusive and
cta_exclusive2 end with every thread reading the per-warp array that they were
given, with no barrier after it, so a store to such an array comes directly
behind a barrier: a warp that has nothing to do in between would else overwrite
what a slower one still reads.  Read from the source; no GPU."""
import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_block_scaled_02_gb300", "csrc",
                      "sample.cu")


def code_lines():
    with open(SOURCE) as f:
        lines = [re.sub(r"//.*", "", line).strip() for line in f]
    return [line for line in lines if line]


def test_arrays_that_sums_read_last_are_written_behind_a_barrier():
    lines = code_lines()
    calls = re.findall(r"cta_exclusive2?<[^;]*?>\(([^;]*?)\);", "\n".join(lines))
    summed = {name for call in calls for name in re.findall(r"sh\.(\w+)", call)}
    assert {"warp_int", "warp_sum"} <= summed               # the pattern finds the calls
    inside = {"warps", "warps_n", "warps_v"}                # their names in the two functions
    stores = [i for i, line in enumerate(lines)
              if any(n in summed | inside for n in re.findall(r"\b(?:sh\.)?(\w+)\[warp\]\s*=[^=]", line))]
    assert len(stores) >= 4
    for i in stores:
        at = i - 1
        while re.fullmatch(r"if \(lane == \d+\) \{", lines[at]):
            at -= 1
        assert lines[at] == "__syncthreads();", lines[i]
