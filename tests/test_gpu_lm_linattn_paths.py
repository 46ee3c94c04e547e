"""GPU tests of linear attention's kernels one by one: cases that the choice of kernel could pass by."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    from sequential_rnn_gb300 import build
    build.build()
    import sequential_rnn_gb300 as S
    return S


def test_zeros_behind_more_than_2_to_the_31_vectors(S):
    """A row of 2^29 + 200 tokens (q, k and v the same for all of them) of which 100 count: the rest of its outputs, more
    16-byte vectors for each CTA than 31 bits hold, are zeros."""
    T, n, Dk, Dv = (1 << 29) + 200, 100, 128, 64
    if torch.cuda.mem_get_info()[0] < 160 << 30:
        pytest.skip("needs 140 GB")
    from sequential_rnn_gb300._lib import rnn_linattn_desc_t, rnn_linattn_strides_t
    q, k, v = (torch.randn(1, 1, 1, D, device="cuda").bfloat16() for D in (Dk, Dk, Dv))
    g = torch.tensor([-0.05], device="cuda")
    desc = rnn_linattn_desc_t(1, T, 1, 1, Dk, Dv, 0.5, 0)
    st = rnn_linattn_strides_t()
    st.o[:] = (Dv, Dv, Dv)
    o = torch.ones(T, 1, 1, Dv, dtype=torch.bfloat16, device="cuda")
    state = torch.empty(1, 1, Dk, Dv, device="cuda")
    ws = torch.empty(S.rnn_linattn_workspace_size(desc, 0), dtype=torch.uint8, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    assert S.rnn_linattn_fwd(desc, st, q, k, v, g, lens, None, o, state, ws) == 0
    assert S.rnn_read_status(ws) == 0
    want = S.linear_attention(*(x.expand(n, 1, 1, x.shape[-1]).contiguous() for x in (q, k, v)), g, scale=0.5)
    assert torch.equal(o[:n], want["o"]) and torch.equal(state, want["state"])
    assert not any(o[lo:lo + (1 << 24)].any().item() for lo in range(n, T, 1 << 24))
    del o, ws
    torch.cuda.empty_cache()


@pytest.mark.parametrize("token", [4, -64])
def test_a_step_does_not_use_token_strides(S, token):
    """A single token has no token stride: any value stands there."""
    from sequential_rnn_gb300._lib import rnn_linattn_desc_t, rnn_linattn_strides_t
    B, NH, D = 3, 2, 64
    q, k, v = (torch.randn(B, NH, D, device="cuda").bfloat16() for _ in range(3))
    g, state = torch.tensor([-0.1, -0.2], device="cuda"), torch.randn(B, NH, D, D, device="cuda")
    st = rnn_linattn_strides_t()
    for n in ("q", "k", "v"):
        getattr(st, n)[:] = (token, NH * D, D)
    st.o[:] = (token, 3, 5)
    o, s = torch.empty_like(v), state.clone()
    assert S.rnn_linattn_step(rnn_linattn_desc_t(1, 1, B, NH, D, D, 0.5, 0), st, q, k, v, g, None, B, s, o) == 0
    want = S.linear_attention_step(q, k, v, g, state, scale=0.5)
    assert torch.equal(o, want) and torch.equal(s, state)
