"""GPU tests of linear attention's kernels one by one: cases that the choice of kernel could pass by.  Each asserts which
kernels its sizes take (`tcgen05`), so that another choice cannot take them out of the tests unseen.

Tolerances as in test_gpu_lm_linattn: bf16 operands (scores times their decay, the state) and the result are rounded
once, 2^-8 of each; sums in fp32, 2^-18 of the magnitudes of all products.  Chunks of 128 tokens on tcgen05, of 64 else.
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import lm_oracle as O
from tests.test_gpu_lm_linattn import close, draw, np64

pytestmark = pytest.mark.gpu
TOKENS = ("q", "k", "v", "do")
# head sizes with lengths from which on tcgen05 takes both passes
WIDE = [(128, 128, 128), (256, 256, 128), (64, 128, 512)]


@pytest.fixture(scope="module")
def S():
    from sequential_rnn_gb300 import build
    build.build()
    import sequential_rnn_gb300 as S
    return S


def tcgen05(S, T, B, NH, Dk, Dv, gradient=False, dtype="bf16"):
    """Whether such a call's kernels are the tcgen05 ones: the others refuse the flag that withholds an arrival (no operand
    is given, so nothing is launched)."""
    from sequential_rnn_gb300._lib import load, rnn_linattn_desc_t
    d = rnn_linattn_desc_t(1 if dtype == "bf16" else 0, T, B, NH, Dk, Dv, 1.0, S.RNN_FLAG_TEST_TIMEOUT)
    f, n = (load().rnn_linattn_bwd, 12) if gradient else (load().rnn_linattn_fwd, 8)
    st = f(ctypes.byref(d), None, *[None] * n, ctypes.c_void_p(256), 1 << 50, None)
    assert st in (1, 2)
    return st == 1


def segments(S, T, B, NH, Dk, Dv, gradient=False):
    """Whether a tcgen05 call cuts the token axis: what its workspace holds beside the chunk states."""
    from sequential_rnn_gb300._lib import rnn_linattn_desc_t
    d = rnn_linattn_desc_t(1, T, B, NH, Dk, Dv, 1.0, 0)
    chunks = -(-T // 128) * B * NH * Dk * Dv * 2 * (3 if gradient else 1)
    return S.rnn_linattn_workspace_size(d, int(gradient)) > 256 + chunks


def size(d):
    return (*d["q"].shape, d["v"].shape[-1])


def forward(S, d, scale=0.37, state=True, chunk=128):
    """Against the oracle; the call's outputs."""
    out = S.linear_attention(d["q"], d["k"], d["v"], d["g"], state=d["s0"] if state else None, lens=d["lens"], scale=scale)
    lens = None if d["lens"] is None else d["lens"].tolist()
    a, s0 = [np64(d[n]) for n in "qkvg"], np64(d["s0"]) if state else None
    o, s = O.linear_attention(*a, s0, lens, scale)
    mag, fin = O.linear_attention_bound(*a, s0, lens, intra=scale, inter=scale, chunk=chunk)
    close(out["o"], o, mag, "bf16", "o")
    close(out["state"], s, (None, fin), "f32", "state")
    return {n: out[n] for n in ("o", "state")}


def backward(S, d, scale=0.37, state=True, chunk=128, chunk_dv=128):
    s0, ds = (d["s0"], d["ds"]) if state else (None, None)
    out = S.linear_attention_backward(d["q"], d["k"], d["v"], d["g"], d["do"], state=s0, dstate=ds, lens=d["lens"],
                                      scale=scale)
    lens = None if d["lens"] is None else d["lens"].tolist()
    q, k, v, g, do, s0, ds = (np64(x) for x in (d["q"], d["k"], d["v"], d["g"], d["do"], s0, ds))
    want = O.linear_attention_backward(q, k, v, g, do, s0, ds, lens, scale)
    t = lambda x: None if x is None else np.swapaxes(x, -1, -2)  # noqa: E731
    mq, _ = O.linear_attention_bound(do, v, k, g, t(s0), lens, intra=scale, inter=scale, chunk=chunk)
    mk, _ = O.linear_attention_bound(v, do, q, g, t(ds), lens, True, scale, 1.0, scale, chunk)
    mv, ms = O.linear_attention_bound(k, q, do, g, ds, lens, True, scale, 1.0, scale, chunk_dv)
    for n, w, m in zip(("dq", "dk", "dv"), want, (mq, mk, mv)):
        close(out[n], w, m, "bf16", n)
    close(out["dstate"], want[3], (None, ms), "f32", "dstate")
    return {n: out[n] for n in ("dq", "dk", "dv", "dstate")}


def both(S, d, **kw):
    assert tcgen05(S, *size(d)) and tcgen05(S, *size(d), gradient=True)
    return {**forward(S, d, **kw), **backward(S, d, **kw)}


def same(a, b):
    return all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("Dk,Dv,T", [(D, E, T + n) for D, E, T in WIDE for n in (0, 1, 12, 63, 64, 127, 128, 129, 200)])
def test_lengths(S, T, Dk, Dv):
    both(S, draw(T, T, 2, 2, Dk, Dv, "bf16"))


@pytest.mark.parametrize("Dk,Dv,T", [(128, 128, 260), (256, 256, 260), (64, 128, 520), (128, 128, 3000), (256, 256, 6000)])
def test_rows_of_every_length_and_values_behind_them(S, Dk, Dv, T):
    """Rows without a token, lens outside [0, T], and NaN / infinity behind a row's last token."""
    lens = [0, 1, 127, 128, 129, 255, 256, 257, T - 1, T, 9 * T, -3] if T < 1000 else [T, T // 3 + 1]
    NH = 2 if T < 1000 else 1
    assert segments(S, T, len(lens), NH, Dk, Dv) == segments(S, T, len(lens), NH, Dk, Dv, True) == (T > 1000)
    d = draw(1, T, len(lens), NH, Dk, Dv, "bf16", lens=lens)
    for b, n in enumerate(lens):
        for name in TOKENS:
            d[name][max(n, 0):, b] = float("nan") if b % 2 else float("inf")
    want = both(S, {n: torch.nan_to_num(x, 0, 0, 0) if n in TOKENS else x for n, x in d.items()})
    got = S.linear_attention(d["q"], d["k"], d["v"], d["g"], state=d["s0"], lens=d["lens"], scale=0.37)
    assert torch.equal(got["o"], want["o"]) and torch.equal(got["state"], want["state"])
    if lens[0] == 0:
        assert torch.equal(got["state"][0], d["s0"][0]) and not got["o"][:, 0].any()
    got = S.linear_attention_backward(d["q"], d["k"], d["v"], d["g"], d["do"], state=d["s0"], dstate=d["ds"],
                                      lens=d["lens"], scale=0.37)
    assert all(torch.equal(got[n], want[n]) for n in ("dq", "dk", "dv", "dstate"))


@pytest.mark.parametrize("Dk,Dv,T,B", [(128, 128, 260, 2), (256, 256, 260, 2), (64, 128, 520, 2), (128, 128, 3000, 1)])
def test_decays(S, Dk, Dv, T, B):
    """No decay, all forgotten at once, and decays whose powers underflow inside a chunk."""
    g = [0.0, -float("inf"), -1e-4, -3.0, -40.0]
    assert segments(S, T, B, len(g), Dk, Dv) == (T > 1000)
    both(S, draw(2, T, B, len(g), Dk, Dv, "bf16", log_decay=g))


@pytest.mark.parametrize("Dk,Dv,T", [(128, 128, 300), (256, 256, 300), (64, 128, 600), (128, 128, 3000)])
def test_no_initial_state_and_default_scale(S, Dk, Dv, T):
    d = draw(3, T, 1, 2, Dk, Dv, "bf16")
    both(S, d, state=False)
    args = (d["q"], d["k"], d["v"], d["g"])
    a, b = (S.linear_attention(*args, **kw)["o"] for kw in ({}, {"scale": Dk ** -0.5}))
    assert torch.equal(a, b)


@pytest.mark.parametrize("Dk,Dv,T", [(128, 128, 300), (256, 256, 300), (64, 128, 600), (128, 128, 3000), (256, 64, 3000)])
def test_the_final_state_over_the_initial_one(S, Dk, Dv, T):
    from sequential_rnn_gb300._lib import rnn_linattn_desc_t
    d = draw(5, T, 1, 2, Dk, Dv, "bf16")
    assert tcgen05(S, *size(d)) and segments(S, *size(d)) == (T > 1000)
    want = S.linear_attention(d["q"], d["k"], d["v"], d["g"], state=d["s0"], scale=0.125)
    desc = rnn_linattn_desc_t(1, T, 1, 2, Dk, Dv, 0.125, 0)
    s, o = d["s0"].clone(), torch.empty_like(d["v"])
    ws = torch.empty(S.rnn_linattn_workspace_size(desc, 0), dtype=torch.uint8, device="cuda")
    assert S.rnn_linattn_fwd(desc, None, d["q"], d["k"], d["v"], d["g"], None, s, o, s, ws) == 0
    assert S.rnn_read_status(ws) == 0
    assert torch.equal(s, want["state"]) and torch.equal(o, want["o"])


@pytest.mark.parametrize("Dk,Dv,T", [(128, 128, 200), (256, 256, 200), (64, 128, 520)])
def test_strided_and_broadcast_operands(S, Dk, Dv, T):
    """Views of one fused projection; keys and values, and the gradient that comes in, that all heads or all rows share."""
    B, NH = 3, 4
    d = draw(6, T, B, NH, Dk, Dv, "bf16", lens=[T, T - 70, 5])
    fused = torch.cat([d[n].flatten(2) for n in TOKENS], -1)
    view, at = {}, 0
    for n in TOKENS:
        w = NH * d[n].shape[-1]
        view[n] = fused[..., at:at + w].unflatten(-1, (NH, -1))
        at += w
    assert not view["q"].is_contiguous()
    assert same(both(S, dict(d, **view)), both(S, d))
    heads = {n: d[n][:, :, :1].expand(d[n].shape) for n in ("k", "v", "do")}
    rows = {n: d[n][:, :1].expand(d[n].shape) for n in ("q", "k", "v")}
    for shared in (heads, rows):
        plain = {n: x.contiguous() for n, x in shared.items()}
        assert same(both(S, dict(d, **shared)), both(S, dict(d, **plain)))


@pytest.mark.parametrize("Dk,Dv,T", [(128, 128, 200), (256, 256, 200), (64, 128, 520), (128, 128, 3000)])
@pytest.mark.parametrize("name", TOKENS)
def test_an_operand_that_all_tokens_share(S, name, Dk, Dv, T):
    """A token stride of zero has no tensor map: such launches (the forward's, which has no do; the gradient's, with unequal
    head sizes one for dq and dk and one for dv, which has no v) go to the mma.sync kernels, whole rows at a time."""
    o = 128 if name == "do" else 64
    dv = 128 if name == "v" and Dk != Dv else 64
    d = draw(7, T, 2, 2, Dk, Dv, "bf16", lens=[T, T - 33])
    d[name] = d[name][:1].expand(d[name].shape)
    assert d[name].stride(0) == 0
    assert tcgen05(S, *size(d)) and tcgen05(S, *size(d), gradient=True)  # but for the stride
    for state in (True, False):
        forward(S, d, state=state, chunk=o)
        backward(S, d, state=state, chunk=64, chunk_dv=dv)


def test_offsets_past_32_bits(S):
    """Token strides that put the last tokens over 2^32 bytes and 2^31 elements into the buffer."""
    T, pitch = 600, 4 << 20
    buf = torch.zeros(T * pitch, dtype=torch.bfloat16, device="cuda")
    d = draw(7, T, 1, 2, 128, 128, "bf16")
    assert tcgen05(S, *size(d)) and tcgen05(S, *size(d), gradient=True)
    far = dict(d)
    for i, n in enumerate(TOKENS):
        far[n] = buf.as_strided(d[n].shape, (pitch, 256, 128, 1), 1024 * i)
        far[n].copy_(d[n])
    call = lambda d: {**S.linear_attention(d["q"], d["k"], d["v"], d["g"], state=d["s0"]),  # noqa: E731
                      **S.linear_attention_backward(d["q"], d["k"], d["v"], d["g"], d["do"], dstate=d["ds"])}
    got, want = call(far), call(d)
    assert all(torch.equal(got[n], want[n]) for n in ("o", "state", "dq", "dk", "dv", "dstate"))


@pytest.mark.parametrize("Dk,Dv,T", [(128, 128, 400), (256, 256, 400), (64, 128, 600), (128, 128, 3000)])
def test_other_stream_graph_and_repeatability(S, Dk, Dv, T):
    d = draw(12, T, 1, 3, Dk, Dv, "bf16")
    assert tcgen05(S, *size(d)) and tcgen05(S, *size(d), gradient=True)
    args, st = (d["q"], d["k"], d["v"], d["g"]), {"state": d["s0"]}
    call = lambda **kw: {**S.linear_attention(*args, **st, **kw),  # noqa: E731
                         **S.linear_attention_backward(*args, d["do"], dstate=d["ds"], **st, **kw)}
    names = ("o", "state", "dq", "dk", "dv", "dstate")
    # (both calls return a workspace under one name; the gradient's initial state is `dstate`)
    want = call()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for handle in (s, s.cuda_stream):
        got = call(stream=handle)
        s.synchronize()
        assert all(torch.equal(got[n], want[n]) for n in names)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(check=False)
    d["v"].copy_(draw(14, T, 1, 3, Dk, Dv, "bf16")["v"])
    graph.replay()
    torch.cuda.synchronize()
    want = call()
    assert all(torch.equal(got[n], want[n]) for n in names)


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


def test_the_shapes_of_values_that_are_not_finite_reach_every_kernel(S):
    from tests.test_gpu_lm_linattn_values import SHAPES
    took = [(tcgen05(S, T, 3, 2, Dk, Dv, dtype=dtype), Dk) for dtype, T, Dk, Dv in SHAPES]
    assert took == [(False, 64), (False, 256), (False, 64), (False, 32), (False, 128), (False, 256), (False, 64),
                    (True, 128), (True, 256), (True, 64), (True, 256), (True, 128)]
    assert segments(S, 3000, 3, 2, 128, 128) and not segments(S, 300, 3, 2, 128, 128)
