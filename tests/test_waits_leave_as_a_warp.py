"""Roles that a whole warp runs leave their loop over bounded waits as a warp: a
lane that gave up alone would leave the others in a shuffle, a vote or a barrier
that waits for it, and a recorded timeout would become a kernel without an end
(CPU only, by reading the sources)."""
import os
import re

import pytest

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "mixed_precision_quantized_act_b200", "csrc")
# a lane's own wait that decides by itself where the lane goes
# or that is the operand of a barrier, which counts whole warps
ALONE = re.compile(r"if \(!mbar_wait\([^;]*\)\)\s*(?:break|return|continue)|while \(!?mbar_wait\(|named_bar_and\([^;]*mbar_wait\(")


# every role of these kernels is a warp's or more
@pytest.mark.parametrize("name", ["kv4_prompt.cuh", "w8a8.cuh"])
def test_no_lane_leaves_alone(name):
    with open(os.path.join(CSRC, name)) as f:
        assert not [m.group(0) for m in ALONE.finditer(f.read())]


def test_the_search_finds_what_it_looks_for():
    assert ALONE.search("if (!mbar_wait(&k_empty[s], phase ^ 1, &abort_flag)) break;")
    assert ALONE.search("if (!named_bar_and(1, 256, mbar_wait(full, parity, abort))) return false;")
    assert not ALONE.search("if (!warp_wait(&k_empty[s], phase ^ 1, &abort_flag)) break;")
    assert not ALONE.search("if (!__all_sync(0xFFFFFFFFu, mbar_wait(&s_full[i][h], phase, &abort_flag))) return;")
