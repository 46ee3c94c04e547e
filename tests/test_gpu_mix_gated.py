"""GPU tests of the gated linear recurrence against the fp64 oracle.  Tolerances are the oracle's bounds of fp32
arithmetic (oracle/mix_oracle.py derives them) plus, for bf16 results, half a step of bf16: 2^-8 of the value."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import mix_oracle as O

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = 2.0 ** -126  # subnormal results lose bits


@pytest.fixture(scope="module")
def S():
    from sequential_rnn_gb300 import build
    build.build()
    import sequential_rnn_gb300 as S
    return S


def np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def rand(seed, *shape, dtype="f32", scale=1.0):
    x = np.random.default_rng(seed).normal(size=shape) * scale
    return torch.from_numpy(np.asarray(x, np.float32)).to("cuda", DT[dtype])


def inputs(T, B, NH, D, gates, dtype, seed=0):
    Wx = rand(seed, T, B, NH, len(gates), D)
    # forget gates from none to a long memory
    Wx[..., gates.index("f"), :] += torch.linspace(-3, 9, D, device="cuda")
    return (Wx.to(DT[dtype]).view(T, B, NH, len(gates) * D), rand(seed + 1, B, NH, D), rand(seed + 2, T, B, NH, D, dtype=dtype),
            rand(seed + 3, B, NH, D))


def close(got, want, err, half=2.0 ** -24):
    got = np64(got)
    tol = err + half * np.abs(want) * (1 + 1e-3) + half * err + TINY
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], tol[bad][:5])


def check(S, T, B, NH, D, gates, dtype, lens=None, state=True, seed=0):
    Wx, s0, dy, ds = inputs(T, B, NH, D, gates, dtype, seed)
    if not state:
        s0 = ds = None
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = S.gated_recurrence(Wx, gates=gates, state=s0, lens=ln, train=True)
    g = S.gated_recurrence_backward(Wx, out["stash"], dy, gates=gates, dstate=ds, lens=ln)
    a = (None if s0 is None else np64(s0), None if ds is None else np64(ds))
    f = O.gated(np64(Wx), gates, a[0], lens, dtype == "bf16")
    b = O.gated_backward(np64(Wx), gates, np64(dy), a[0], a[1], lens, dtype == "bf16")
    close(out["y"], f["y"], f["y_err"], HALF[dtype])
    close(out["state"], f["state"], f["state_err"])
    close(g["dWx"], b["dWx"], b["dWx_err"], HALF[dtype])
    close(g["dstate"], b["dstate"], b["dstate_err"])
    alone = S.gated_recurrence(Wx, gates=gates, state=s0, lens=ln)
    assert "stash" not in alone and torch.equal(alone["y"], out["y"]) and torch.equal(alone["state"], out["state"])


# lengths around a run (8), a round (64) and several rounds of a cluster; sizes on tiles of 64 and 32 channels, with idle lanes,
# and value by value
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gates", ["fz", "fzo", "ifzo"])
@pytest.mark.parametrize("T,B,NH,D", [(1, 1, 1, 1), (0, 2, 3, 8), (7, 2, 2, 33), (8, 3, 1, 64), (9, 1, 5, 40), (64, 2, 2, 32),
                                      (65, 1, 1, 130), (200, 3, 2, 31), (1100, 2, 3, 64), (700, 1, 1, 6),
                                      (32, 2, 2, 8), (100, 4, 3, 136), (2500, 1, 1, 48), (257, 30, 8, 72),
                                      (1500, 1, 2, 64), (129, 40, 6, 32), (5000, 1, 1, 96), (65, 3, 2, 64)])
def test_shapes(S, T, B, NH, D, gates, dtype):
    check(S, T, B, NH, D, gates, dtype, seed=T + D)


@pytest.mark.parametrize("gates", ["fz", "fzo", "ifzo"])
@pytest.mark.parametrize("T,lens", [(70, [70, 0, 1, 69, 64, 1000, -5]), (1200, [1200, 3, 513, 0, 8, 1025, 72])])
def test_lengths(S, T, lens, gates):
    check(S, T, len(lens), 2, 32, gates, "bf16", lens=lens)
    check(S, T, len(lens), 1, 5, gates, "f32", lens=lens, state=False)


def test_wide_rows_take_one_cta_each(S):
    """Enough tiles that no cluster is formed."""
    check(S, 150, 40, 12, 64, "fz", "bf16")


@pytest.mark.parametrize("gates", ["fz", "ifzo"])
def test_constant_gates_keep_a_long_memory(S, gates):
    """A forget gate of 8 in every token: the state after 4000 tokens is as far off as the bound says."""
    T, D = 4000, 64
    Wx, s0, _, _ = inputs(T, 1, 1, D, gates, "f32", 3)
    Wx.view(T, len(gates), D)[:, gates.index("f")] = 8.0
    out = S.gated_recurrence(Wx, gates=gates, state=s0)
    f = O.gated(np64(Wx), gates, np64(s0))
    close(out["state"], f["state"], f["state_err"])


@pytest.mark.parametrize("D", [32, 64, 33])
@pytest.mark.parametrize("gates", ["fz", "ifzo"])
def test_dead_tokens_do_not_matter(S, gates, D):
    T, B, NH, lens = 100, 3, 2, [0, 50, 67]
    Wx, s0, dy, ds = inputs(T, B, NH, D, gates, "bf16")
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    bad, bady = Wx.clone(), dy.clone()
    for b, n in enumerate(lens):
        for i, v in enumerate((float("nan"), float("inf"), -float("inf"), torch.finfo(torch.bfloat16).min)):
            bad[n + i::4, b] = v
            bady[n + i::4, b] = v
    res = []
    for w, d in ((Wx, dy), (bad, bady)):
        out = S.gated_recurrence(w, gates=gates, state=s0, lens=ln, train=True)
        g = S.gated_recurrence_backward(w, out["stash"], d, gates=gates, dstate=ds, lens=ln)
        res.append((out["y"], out["state"], g["dWx"], g["dstate"]))
    for a, b in zip(*res):
        assert torch.equal(a, b)
    assert (res[1][0][67:] == 0).all() and (res[1][2][67:] == 0).all()
    assert torch.equal(res[1][1][0], s0[0]) and torch.equal(res[1][3][0], ds[0])


@pytest.mark.parametrize("D", [32, 33])  # on tiles, and value by value
def test_values_that_are_not_finite_stay_in_their_channel(S, D):
    T, B, NH = 150, 2, 1
    Wx, s0, dy, ds = inputs(T, B, NH, D, "fz", "f32")
    Wx.view(T, B, 2, D)[..., 0, :].clamp_(-3, 3)
    bad = Wx.clone()
    bad[70, 0, 0, D + 3] = float("inf")   # z
    bad[20, 1, 0, 7] = float("nan")       # f
    a, b = (S.gated_recurrence(w, state=s0) for w in (Wx, bad))
    same = torch.ones_like(a["y"], dtype=torch.bool)
    same[70:, 0, 0, 3] = False
    same[20:, 1, 0, 7] = False
    assert torch.equal(a["y"][same], b["y"][same])
    assert torch.isinf(b["y"][70:, 0, 0, 3]).all() and torch.isnan(b["y"][20:, 1, 0, 7]).all()
    # gates at the ends: all forgotten, all kept
    Wx.view(T, B, 2, D)[:, :, 0, :5] = -float("inf")
    Wx.view(T, B, 2, D)[:, :, 0, 5:9] = float("inf")
    y = S.gated_recurrence(Wx, state=s0)["y"][:, :, 0]
    assert torch.equal(y[..., :5], Wx.view(T, B, 2, D)[:, :, 1, :5])
    assert torch.equal(y[..., 5:9], s0[:, 0, 5:9].expand(T, B, 4))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gates", ["fz", "fzo", "ifzo"])
@pytest.mark.parametrize("B,NH,D", [(1, 1, 1), (16, 12, 64), (5, 3, 33), (70, 4, 256)])
def test_step(S, B, NH, D, gates, dtype):
    Wx, _, _, _ = inputs(1, B, NH, D, gates, dtype)
    cache = rand(9, B + 3, NH, D)
    slots = torch.randperm(B + 3, generator=torch.Generator().manual_seed(1))[:B].int().cuda()
    if B > 3:
        slots[1], slots[3] = -1, B + 3  # rows without a state
    old = cache.clone()
    y = S.gated_recurrence_step(Wx[0], cache, gates=gates, slots=slots)
    ok = [(b, int(s)) for b, s in enumerate(slots) if 0 <= s < B + 3]
    at = [s for _, s in ok]
    f = O.gated(np64(Wx)[:, [b for b, _ in ok]], gates, np64(old)[at], fast=dtype == "bf16")
    close(cache[at], f["state"], f["state_err"])
    close(y[[b for b, _ in ok]], f["y"][0], f["y_err"][0], HALF[dtype])
    rest = [s for s in range(B + 3) if s not in at]
    assert torch.equal(cache[rest], old[rest])
    if B > 3:
        assert (y[1] == 0).all() and (y[3] == 0).all()
    # without slots: row b's state is b
    cache2 = old[:B].clone()
    y2 = S.gated_recurrence_step(Wx[0], cache2, gates=gates)
    f = O.gated(np64(Wx), gates, np64(old[:B]), fast=dtype == "bf16")
    close(cache2, f["state"], f["state_err"])
    close(y2, f["y"][0], f["y_err"][0], HALF[dtype])


def test_steps_continue_a_prompt(S):
    Wx, s0, _, _ = inputs(40, 3, 2, 32, "ifzo", "bf16")
    want = S.gated_recurrence(Wx, gates="ifzo", state=s0)
    out = S.gated_recurrence(Wx[:25], gates="ifzo", state=s0)
    state, ys = out["state"], [out["y"]]
    for t in range(25, 40):
        ys.append(S.gated_recurrence_step(Wx[t], state, gates="ifzo")[None])
    f = O.gated(np64(Wx), "ifzo", np64(s0), fast=True)
    close(torch.cat(ys), f["y"], f["y_err"], HALF["bf16"])
    close(state, f["state"], f["state_err"])
    close(want["state"], f["state"], f["state_err"])


@pytest.mark.parametrize("T", [30, 130])  # 130: the aligned ones run on tiles
def test_unaligned_views(S, T):
    """Contiguous tensors that begin at an odd element; a stash of the one form in the other's gradient."""
    B, NH, D = 2, 1, 32
    Wx, s0, dy, ds = inputs(T, B, NH, D, "fz", "bf16")
    buf = torch.empty(Wx.numel() + 1, dtype=torch.bfloat16, device="cuda")
    odd = buf[1:].view(Wx.shape).copy_(Wx)
    a = S.gated_recurrence(Wx, state=s0, train=True)
    b = S.gated_recurrence(odd, state=s0, train=True)
    f = O.gated(np64(Wx), "fz", np64(s0), fast=True)
    for o in (a, b):
        close(o["y"], f["y"], f["y_err"], HALF["bf16"])
    g = O.gated_backward(np64(Wx), "fz", np64(dy), np64(s0), np64(ds), fast=True)
    for w, stash in ((odd, b["stash"]), (odd, a["stash"]), (Wx, b["stash"])):
        r = S.gated_recurrence_backward(w, stash, dy, dstate=ds)
        close(r["dWx"], g["dWx"], g["dWx_err"], HALF["bf16"])
        close(r["dstate"], g["dstate"], g["dstate_err"])


def test_in_place_states_and_streams(S):
    """stateT in state0's place; a call on a side stream; the same result every time."""
    T, B, NH, D = 600, 2, 3, 64
    Wx, s0, dy, ds = inputs(T, B, NH, D, "fzo", "bf16")
    want = S.gated_recurrence(Wx, gates="fzo", state=s0, train=True)
    from sequential_rnn_gb300._lib import rnn_gated_desc_t
    d = rnn_gated_desc_t(1, T, B, NH, D, 3, 0)
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")  # (a call clears its status word)
    y, st = torch.empty_like(want["y"]), s0.clone()
    assert S.rnn_gated_fwd(d, Wx, None, st, y, st, None, ws) == 0 and S.rnn_read_status(ws) == 0
    assert torch.equal(y, want["y"]) and torch.equal(st, want["state"])
    g = S.gated_recurrence_backward(Wx, want["stash"], dy, gates="fzo", dstate=ds)
    dW, dst = torch.empty_like(Wx), ds.clone()
    assert S.rnn_gated_bwd(d, Wx, None, want["stash"], dy, dst, dW, dst, ws) == 0 and S.rnn_read_status(ws) == 0
    assert torch.equal(dW, g["dWx"]) and torch.equal(dst, g["dstate"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = S.gated_recurrence(Wx, gates="fzo", state=s0, stream=side)
    side.synchronize()
    assert torch.equal(out["y"], want["y"])
    assert ctypes.sizeof(rnn_gated_desc_t) == 28


def test_captured_calls(S):
    """Forward, backward and a step in one graph, replayed on other inputs."""
    T, B, NH, D = 300, 2, 2, 64
    Wx, s0, dy, ds = inputs(T, B, NH, D, "ifzo", "bf16")
    cache = s0.clone()

    def step():
        o = S.gated_recurrence(Wx, gates="ifzo", state=s0, train=True, check=False)
        g = S.gated_recurrence_backward(Wx, o["stash"], dy, gates="ifzo", dstate=ds, check=False)
        return o["y"], g["dWx"], g["dstate"], S.gated_recurrence_step(Wx[0], cache, gates="ifzo")

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    new = inputs(T, B, NH, D, "ifzo", "bf16", seed=50)
    for x, y in zip((Wx, s0, dy, ds), new):
        x.copy_(y)
    cache.copy_(s0)
    graph.replay()
    torch.cuda.synchronize()
    first = cache.clone()
    cache.copy_(s0)
    for a, b in zip(got, step()):
        assert torch.equal(a, b)
    assert torch.equal(first, cache)


@pytest.mark.parametrize("B", [1, 40])  # a cluster for each tile, and a CTA
def test_an_expired_wait_is_reported(S, B):
    """RNN_FLAG_TEST_TIMEOUT: no tile is brought, every wait runs out after 50 ms; the next call is fine."""
    from sequential_rnn_gb300._lib import RNN_FLAG_TEST_TIMEOUT, rnn_gated_desc_t
    T, NH, D = 1000, 12, 64
    Wx, s0, dy, ds = inputs(T, B, NH, D, "fz", "bf16")
    want = S.gated_recurrence(Wx, state=s0, train=True)
    d = rnn_gated_desc_t(1, T, B, NH, D, 2, RNN_FLAG_TEST_TIMEOUT)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    y, dW, st = torch.empty_like(want["y"]), torch.empty_like(Wx), torch.empty_like(s0)
    assert S.rnn_gated_fwd(d, Wx, None, s0, y, st, None, ws) == 0 and S.rnn_read_status(ws) == 5
    assert S.rnn_gated_bwd(d, Wx, None, want["stash"], dy, ds, dW, st, ws) == 0 and S.rnn_read_status(ws) == 5
    again = S.gated_recurrence(Wx, state=s0, train=True)
    for k in ("y", "state", "stash"):
        assert torch.equal(again[k], want[k])


def test_refusals(S):
    Wx, s0, dy, ds = inputs(4, 2, 2, 8, "fz", "bf16")
    for kw, e in ((dict(gates="fi"), ValueError), (dict(gates=2), TypeError), (dict(gates="fzo"), ValueError),
                  (dict(state=s0[:1]), ValueError), (dict(state=s0.bfloat16()), TypeError),
                  (dict(lens=torch.zeros(2, device="cuda")), TypeError),
                  (dict(lens=torch.zeros(3, dtype=torch.int32, device="cuda")), ValueError)):
        with pytest.raises(e):
            S.gated_recurrence(Wx, **kw)
    with pytest.raises(TypeError):
        S.gated_recurrence(Wx.half())
    with pytest.raises(ValueError, match="contiguous"):
        S.gated_recurrence(Wx.transpose(0, 1))
    with pytest.raises(ValueError):
        S.gated_recurrence(Wx[0])
    out = S.gated_recurrence(Wx, train=True)
    with pytest.raises(ValueError):
        S.gated_recurrence_backward(Wx, out["stash"][:-1], dy)
    with pytest.raises(ValueError):
        S.gated_recurrence_backward(Wx, out["stash"], dy[:-1])
    with pytest.raises(S.RnnError):
        S.gated_recurrence_step(Wx[0], s0[:1])  # fewer states than rows
    with pytest.raises(ValueError):
        S.gated_recurrence_step(Wx[0], s0[..., :4])
    empty = S.gated_recurrence(Wx[:, :0], train=True)
    assert empty["y"].shape == (4, 0, 2, 8) and empty["stash"].numel() == 0
