"""What the kernels' sources keep to where a fault would depend on timing, so that no run shows it reliably."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_deltanet_linear_core_gb300", "csrc")


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", ["attn_tc.cu", "attn_shared_tc.cu"])
def test_the_flag_of_odd_values_is_cleared_behind_a_barrier(name):
    """Every softmax warp reads the flag at the end of a segment, one thread clears it: between the two they meet."""
    text = code(name)
    reads = [m.end() for m in re.finditer(r"= \*odd_v != 0;", text)]
    clears = [m.start() for m in re.finditer(r"\*odd_v = 0;", text)]
    assert len(reads) == 1 and len(clears) == 2  # the first clear comes before any segment
    assert clears[0] < reads[0] < clears[1]
    assert re.search(r"softmax_sync(<NSOFT>)?\(\);", text[reads[0]:clears[1]])


@pytest.mark.parametrize("name", sorted(os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cu*"))))
def test_loads_from_tensor_memory_wait_in_their_own_statement(name):
    """Between two statements the compiler may move or use a register that does not have its value yet."""
    for statement in re.findall(r"asm volatile\((.*?)\);", code(name), re.S):
        loads = [m.start() for m in re.finditer(r"tcgen05\.ld\b", statement)]
        waits = [m.start() for m in re.finditer(r"tcgen05\.wait::ld", statement)]
        assert bool(loads) == bool(waits) and (not loads or loads[-1] < waits[-1])
        if len(loads) > 1:  # a later load's address is not where an earlier one's values go
            assert '"=&r"(r[0])' in statement
