"""Code rules and refusals of the gated recurrence and the clipping that need no GPU."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sequential_rnn_gb300", "csrc")


@pytest.mark.parametrize("name", ["gated.cu", "gated_tile.cu"])
def test_aligned_barriers_follow_a_joined_warp(name):
    """cluster_sync, bar_sync and bar_arrive are barriers of the aligned form, which a warp has to reach with its lanes together:
    what stands directly before each of them joins the lanes, whatever branches came earlier."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    code = re.sub(r"__device__ __forceinline__ void bar_arrive\([^}]*}", "", code)  # its definition
    calls = [m.start() for m in re.finditer(r"\b(cluster_sync|bar_sync|bar_arrive)\(", code)]
    assert len(calls) >= 3
    for at in calls:
        before = re.sub(r"if \((p\.)?cs > 1\)( {)?\s*$", "", code[:at].rstrip()).rstrip()  # (the same for all of a CTA)
        assert before.endswith(("__syncwarp();", "__syncthreads();")), code[max(0, at - 200):at + 40]
