"""GPU tests of what linear attention's tcgen05 kernels do when a wait on the device runs out.

With the descriptor's RNN_FLAG_TEST_TIMEOUT one arrival of each kernel is left out and the waits end after 50 ms: the
other roles give up, what was issued ends, the tensor memory is freed, the kernels return, and the status word tells.
"""
import time

import pytest
import torch

pytestmark = pytest.mark.gpu
RNN_BF16, RNN_ERR_UNSUPPORTED, RNN_ERR_TIMEOUT = 1, 2, 5


@pytest.fixture(scope="module")
def S():
    from sequential_rnn_gb300 import build
    build.build()
    import sequential_rnn_gb300 as S
    return S


def draw(T, B, NH, Dk, Dv):
    g = torch.Generator(device="cuda").manual_seed(T)
    f = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    return (f(T, B, NH, Dk), f(T, B, NH, Dk), f(T, B, NH, Dv), f(T, B, NH, Dv),
            torch.tensor([-0.1, -0.01, -0.5, -1.0], device="cuda")[:NH].contiguous())


def call(S, flags, T, B, NH, Dk, Dv, gradient, lens=None):
    from sequential_rnn_gb300._lib import rnn_linattn_desc_t
    q, k, v, do, g = draw(T, B, NH, Dk, Dv)
    desc = rnn_linattn_desc_t(RNN_BF16, T, B, NH, Dk, Dv, 0.5, flags)
    ws = torch.zeros(S.rnn_linattn_workspace_size(desc, int(gradient)), dtype=torch.uint8, device="cuda")
    state = torch.zeros(B, NH, Dk, Dv, device="cuda")
    lens = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    if gradient:
        out = [torch.zeros_like(x) for x in (q, k, v)]
        st = S.rnn_linattn_bwd(desc, None, q, k, v, g, lens, None, do, None, *out, state, ws)
    else:
        out = [torch.zeros_like(v)]
        st = S.rnn_linattn_fwd(desc, None, q, k, v, g, lens, None, *out, state, ws)
    assert st in (0, RNN_ERR_UNSUPPORTED)
    return st or S.rnn_read_status(ws), out + [state]


@pytest.mark.parametrize("gradient", [False, True])
@pytest.mark.parametrize("T,B,NH,Dk,Dv,lens", [
    (300, 2, 2, 128, 128, None), (300, 3, 2, 128, 128, [300, 0, 131]), (300, 2, 2, 256, 256, None),
    (600, 2, 2, 64, 128, None), (600, 2, 4, 256, 64, [600, 37]), (3000, 1, 1, 128, 128, None),
    (1500, 8, 4, 128, 128, None)])
def test_a_wait_that_runs_out(S, T, B, NH, Dk, Dv, lens, gradient):
    if gradient and Dk > Dv:
        Dk = Dv = 256
    st, want = call(S, 0, T, B, NH, Dk, Dv, gradient, lens)
    assert st == 0
    t0 = time.perf_counter()
    st, _ = call(S, S.RNN_FLAG_TEST_TIMEOUT, T, B, NH, Dk, Dv, gradient, lens)
    assert st == RNN_ERR_TIMEOUT and time.perf_counter() - t0 < 5
    st, got = call(S, 0, T, B, NH, Dk, Dv, gradient, lens)  # the next call is not touched by it
    assert st == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


def test_kernels_without_waits_refuse(S):
    for T, D in ((64, 64), (64, 128)):
        assert call(S, S.RNN_FLAG_TEST_TIMEOUT, T, 2, 2, D, D, False)[0] == RNN_ERR_UNSUPPORTED
        assert call(S, S.RNN_FLAG_TEST_TIMEOUT, T, 2, 2, D, D, True)[0] == RNN_ERR_UNSUPPORTED
