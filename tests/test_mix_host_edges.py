"""Code rules and refusals of the gated recurrence and the clipping that need no GPU."""
import ctypes
import os
import re

import pytest

from tests.test_mix_host import A, INF, P, W, clip, gated, gdesc, lib  # noqa: F401 (lib: the fixture)

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


def test_clip_counts_that_pass_32_bits(lib):  # noqa: F811
    """Units of 16 KB are counted in 32 bits, over all tensors of a call: each launch's partial sums have their place in the
    workspace, whose size follows from the tensors' number alone."""
    most = (1 << 40) // 4096 * 4096  # 2^28 units of fp32
    for n in (8, 16, 17, 256):
        tensors = [A + i * (most * 4) for i in range(n)]
        assert clip(lib, tensors, sizes=[most] * n, limit=1.0) == 2, n
        assert clip(lib, [A] * n, sizes=[most] * n, limit=INF) == 2, n
    lot = (1 << 28) + 1
    assert lib.rnn_clip_grad_norm_workspace_size(lot - 1) > 0
    assert lib.rnn_clip_grad_norm_workspace_size(lot) == lib.rnn_clip_grad_norm_workspace_size((1 << 31) - 1) == 0
    assert lib.rnn_clip_grad_norm(lot, P(A), P(A), P(A), 1.0, None, P(W), 1 << 40, None) == 2


@pytest.mark.parametrize("kw", [dict(dtype=2), dict(T=-1), dict(D=0), dict(gates=1), dict(gates=5), dict(flags=1)])
def test_gated_config_refusals(lib, kw):  # noqa: F811
    out = (ctypes.c_int32 * 7)(*[9] * 7)
    assert lib.rnn_gated_config(ctypes.byref(gdesc(**kw)), 0, out) == 1 and list(out) == [9] * 7
    assert lib.rnn_gated_config(None, 0, out) == lib.rnn_gated_config(ctypes.byref(gdesc()), 0, None) == 1
    for none in (dict(B=0), dict(NH=0)):
        assert lib.rnn_gated_config(ctypes.byref(gdesc(**none)), 1, out) == 0 and list(out) == [0] * 7


def test_the_timeout_flag_is_refused_where_no_tile_is_brought(lib):  # noqa: F811
    for call, names in (("fwd", ("Wx", "y")), ("bwd", ("Wx", "dy", "dWx"))):
        for n in names:
            assert gated(lib, call, gdesc(T=100, flags=1 << 30), **{n: A + 2}) == 2, (call, n)
    assert gated(lib, "fwd", gdesc(T=100, flags=1 << 30), stash=A + 4) == 2
    assert gated(lib, "bwd", gdesc(T=100, flags=1 << 30), stash=A + 4) == 2
