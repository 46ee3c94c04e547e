"""Refusals of the language-model operators that need no GPU, at the ends of what they take: operands that one pass reads
while another writes them, sizes whose counts pass 32 bits.  Pointers are fake and never dereferenced."""
import ctypes

import pytest

P = ctypes.c_void_p
A, W = 0x10000, 0x20000


@pytest.fixture(scope="module")
def lib():
    from sequential_rnn_gb300 import _lib, build
    build.build()
    return _lib.load()


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (64, 128)])
@pytest.mark.parametrize("state", ["state0", "dstateT"])
def test_linattn_gradient_of_the_state_over_a_state_that_is_read(lib, Dk, Dv, state):
    from sequential_rnn_gb300._lib import rnn_linattn_desc_t
    d = rnn_linattn_desc_t(1, 8, 2, 2, Dk, Dv, 1.0, 0)
    s0, dsT = (A, 0) if state == "state0" else (0, A)
    assert lib.rnn_linattn_bwd(ctypes.byref(d), None, P(A), P(A), P(A), P(A), None, P(s0), P(A), P(dsT), P(A), P(A), P(A),
                               P(A), P(W), 1 << 30, None) == 1


MOST = (1 << 31) - 4096  # columns whose rounding up to tiles and strides over blocks stays within 32 bits


@pytest.mark.parametrize("N", [MOST + 1, (1 << 31) - 128, (1 << 31) - 1])
def test_rows_wider_than_32_bit_counts_are_refused(lib, N):
    assert lib.rnn_rms_norm(1, 1, N, 1e-6, P(A), None, P(A), None, P(A), None, None, None) == 2
    assert lib.rnn_rms_norm_bwd(1, 1, N, P(A), P(A), P(A), P(A), None, P(A), None, None, 0, None) == 2
    assert lib.rnn_quantize_weight(1, 8, N, P(A), P(A), P(A), None) == 2


@pytest.mark.parametrize("N,K", [((1 << 31) - 8, 16), (MOST + 8, 16), (8, (1 << 31) - 16), (8, MOST + 16)])
@pytest.mark.parametrize("M", [1, 65])
def test_projections_wider_than_32_bit_counts_are_refused(lib, M, N, K):
    assert lib.rnn_input_proj_fp8(M, N, K, P(A), P(A), P(A), P(A), None, P(A), P(W), 256, None) == 2
