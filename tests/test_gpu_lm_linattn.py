"""GPU tests of linear attention with a decay for each head, against the fp64 oracle.

Tolerances, from the arithmetic.  bf16: the scores times their decay and the state as an
operand are rounded once (2^-8 of each term: half of the spacing of 8-bit significands; so 2^-8 of the
sum of the terms' magnitudes inside a chunk of 64, which the oracle gives) and the result once (2^-8
of it).  fp32 sums (the states, and the fp32 path): 2^-18 of the sum of magnitudes of all products.
"""
import numpy as np
import pytest
import torch

from oracle import lm_oracle as O

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
H, U = 2.0 ** -8, 2.0 ** -18


@pytest.fixture(scope="module")
def S():
    from sequential_rnn_gb300 import build
    build.build()
    import sequential_rnn_gb300 as S
    return S


def np64(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def draw(seed, T, B, NH, Dk, Dv, dtype, log_decay=None, lens=None):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    f = lambda *s, d="f32", c=1.0: (torch.randn(s, generator=g, device="cuda") * c).to(DT[d])  # noqa: E731
    ld = torch.log1p(-torch.exp2(-torch.linspace(1, 9, NH, device="cuda"))) if log_decay is None else \
        torch.tensor(log_decay, dtype=torch.float32, device="cuda")
    return dict(q=f(T, B, NH, Dk, d=dtype), k=f(T, B, NH, Dk, d=dtype, c=Dk ** -0.5), v=f(T, B, NH, Dv, d=dtype),
                g=ld, do=f(T, B, NH, Dv, d=dtype), s0=f(B, NH, Dk, Dv), ds=f(B, NH, Dk, Dv),
                lens=None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda"))


def close(got, want, mag, dtype, what):
    """mag: magnitudes of the terms that bf16 operands round, and of all products."""
    got = np64(got)
    tol = U * mag[1] + (H * (np.abs(want) + mag[0]) * (1 + H) if dtype == "bf16" else 0.0)
    bad = ~(np.abs(got - want) <= tol + 1e-30)
    assert not bad.any(), (what, int(bad.sum()), float(np.abs(got - want)[bad].max()))


def check_forward(S, d, dtype, scale=0.37, state=True, **kw):
    s0 = d["s0"] if state else None
    out = S.linear_attention(d["q"], d["k"], d["v"], d["g"], state=s0, lens=d["lens"], scale=scale, **kw)
    lens = None if d["lens"] is None else d["lens"].tolist()
    a = [np64(d[n]) for n in ("q", "k", "v", "g")]
    o, s = O.linear_attention(*a, np64(s0), lens, scale)
    mag, fin = O.linear_attention_bound(*a, np64(s0), lens, intra=scale, inter=scale)
    close(out["o"], o, mag, dtype, "o")
    close(out["state"], s, (None, fin), "f32", "state")
    return out


def check_backward(S, d, dtype, scale=0.37, state=True):
    s0, ds = (d["s0"], d["ds"]) if state else (None, None)
    out = S.linear_attention_backward(d["q"], d["k"], d["v"], d["g"], d["do"], state=s0, dstate=ds,
                                      lens=d["lens"], scale=scale)
    lens = None if d["lens"] is None else d["lens"].tolist()
    q, k, v, g, do = (np64(d[n]) for n in ("q", "k", "v", "g", "do"))
    s0, ds = np64(s0), np64(ds)
    want = O.linear_attention_backward(q, k, v, g, do, s0, ds, lens, scale)
    t = lambda x: None if x is None else np.swapaxes(x, -1, -2)  # noqa: E731
    mq, _ = O.linear_attention_bound(do, v, k, g, t(s0), lens, intra=scale, inter=scale)
    mk, _ = O.linear_attention_bound(v, do, q, g, t(ds), lens, True, scale, 1.0, scale)
    mv, ms = O.linear_attention_bound(k, q, do, g, ds, lens, True, scale, 1.0, scale)
    for n, w, m in zip(("dq", "dk", "dv"), want, (mq, mk, mv)):
        close(out[n], w, m, dtype, n)
    close(out["dstate"], want[3], (None, ms), "f32", "dstate")
    return out


LENGTHS = [1, 2, 31, 32, 33, 63, 64, 65, 127, 129, 200]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", LENGTHS)
def test_lengths(S, T, dtype):
    d = draw(T, T, 2, 3, 64, 64, dtype)
    check_forward(S, d, dtype)
    check_backward(S, d, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Dk,Dv", [(32, 32), (32, 64), (32, 256), (64, 32), (64, 128), (128, 32), (128, 64), (128, 128),
                                   (256, 32), (256, 64), (256, 256)])
def test_head_sizes(S, Dk, Dv, dtype):
    d = draw(Dk + Dv, 150, 2, 2, Dk, Dv, dtype, lens=[150, 77])
    check_forward(S, d, dtype)
    check_backward(S, d, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_of_every_length_and_values_behind_them(S, dtype):
    """Rows without a token, lens outside [0, T], and NaN / infinity behind a row's last token."""
    T, lens = 140, [0, 1, 64, 65, 139, 140, 500, -3]
    d = draw(1, T, len(lens), 2, 64, 64, dtype, lens=lens)
    for b, n in enumerate(lens):
        for name in ("q", "k", "v", "do"):
            d[name][max(n, 0):, b] = float("nan") if b % 2 else float("inf")
    clean = {n: torch.nan_to_num(x, 0, 0, 0) if n in ("q", "k", "v", "do") else x for n, x in d.items()}
    out = S.linear_attention(d["q"], d["k"], d["v"], d["g"], state=d["s0"], lens=d["lens"])
    same = check_forward(S, clean, dtype, scale=64 ** -0.5)
    assert torch.equal(out["o"], same["o"]) and torch.equal(out["state"], same["state"])
    assert torch.equal(out["state"][0], d["s0"][0]) and not out["o"][:, 0].any()
    got = S.linear_attention_backward(d["q"], d["k"], d["v"], d["g"], d["do"], state=d["s0"], dstate=d["ds"],
                                      lens=d["lens"], scale=0.37)
    same = check_backward(S, clean, dtype)
    for n in ("dq", "dk", "dv", "dstate"):
        assert torch.equal(got[n], same[n]), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decays(S, dtype):
    """No decay, all forgotten at once, and decays whose powers underflow inside a chunk."""
    d = draw(2, 130, 2, 5, 64, 64, dtype, log_decay=[0.0, -float("inf"), -1e-4, -3.0, -40.0])
    check_forward(S, d, dtype)
    check_backward(S, d, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_initial_state_and_default_scale(S, dtype):
    d = draw(3, 100, 2, 2, 64, 64, dtype)
    check_forward(S, d, dtype, state=False)
    check_backward(S, d, dtype, state=False)
    a = S.linear_attention(d["q"], d["k"], d["v"], d["g"])["o"]
    b = S.linear_attention(d["q"], d["k"], d["v"], d["g"], scale=0.125)["o"]
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,T,B,NH,Dk,Dv", [("bf16", 3000, 1, 2, 64, 64), ("bf16", 1999, 2, 2, 128, 128),
                                                ("bf16", 1500, 1, 1, 256, 256), ("bf16", 1500, 2, 3, 32, 64),
                                                ("f32", 1500, 1, 2, 64, 64), ("f32", 700, 1, 1, 256, 128)])
def test_long_rows_in_segments(S, dtype, T, B, NH, Dk, Dv):
    """Few heads and many chunks: the token axis is split over the GPU."""
    lens = [T] if B == 1 else [T, T // 3]
    d = draw(4, T, B, NH, Dk, Dv, dtype, lens=lens)
    check_forward(S, d, dtype)
    check_backward(S, d, dtype)


@pytest.mark.parametrize("T,B,NH,Dk,Dv,ragged", [(3001, 8, 4, 256, 256, False), (3001, 8, 4, 256, 256, True),
                                                  (2000, 8, 2, 256, 64, True), (4000, 8, 6, 128, 128, True),
                                                  (4000, 8, 6, 128, 64, False), (4096, 8, 12, 64, 64, True),
                                                  (3000, 8, 4, 128, 256, True), (4000, 8, 4, 64, 256, False),
                                                  (4100, 8, 6, 64, 128, False)])
def test_many_tiles_per_cta(S, T, B, NH, Dk, Dv, ragged):
    """Enough rows and chunks that every CTA of a persistent grid takes several: against the fp32 path (itself
    tested against the oracle) on the same inputs.  Two roundings of operands or result, each uniform within 2^-8 of
    the value (2^-8 / sqrt 3 root mean square): together below 2^-8 of the norm."""
    lens = [T - (T * b) // (B - 1) for b in range(B)] if ragged else None
    d = draw(T + Dk, T, B, NH, Dk, Dv, "bf16", lens=lens)
    f = {n: x.float() if n in ("q", "k", "v", "do") else x for n, x in d.items()}
    got, want = ({**S.linear_attention(x["q"], x["k"], x["v"], x["g"], state=x["s0"], lens=x["lens"]),
                  **{n: t for n, t in S.linear_attention_backward(
                      x["q"], x["k"], x["v"], x["g"], x["do"], state=x["s0"], dstate=x["ds"],
                      lens=x["lens"]).items() if n != "workspace"}} for x in (d, f))
    for n, tol in (("o", H), ("dq", H), ("dk", H), ("dv", H), ("state", 4 * U), ("dstate", 4 * U)):
        a, b = got[n].double(), want[n].double()
        for row in range(B):   # a wrong tile shows in its row
            i = (slice(None), row) if n in ("o", "dq", "dk", "dv") else row
            assert (a[i] - b[i]).norm() <= tol * b[i].norm(), (n, row)


@pytest.mark.parametrize("T,B,NH,Dk,Dv", [(300, 3, 2, 64, 128), (300, 3, 2, 64, 256), (300, 3, 2, 128, 64),
                                          (300, 3, 2, 256, 64), (1030, 8, 12, 64, 64), (1025, 13, 5, 64, 128)])
def test_unequal_head_sizes_and_many_heads(S, T, B, NH, Dk, Dv):
    """The lengths and numbers of heads from which on other kernels take 64 columns, with ragged rows."""
    d = draw(T + Dk + Dv, T, B, NH, Dk, Dv, "bf16", lens=[T, 129, 0] + [T - 7 * b for b in range(B - 3)])
    check_forward(S, d, "bf16")
    if T < 1000:
        check_backward(S, d, "bf16")


@pytest.mark.parametrize("T,B,NH,Dk,Dv", [(150, 19, 12, 64, 64), (150, 20, 12, 64, 64), (150, 38, 2, 64, 64),
                                          (150, 39, 2, 128, 64), (70, 19, 4, 128, 128), (70, 10, 4, 256, 64)])
def test_numbers_of_heads(S, T, B, NH, Dk, Dv):
    """Both sides of the numbers of heads at which a CTA takes more columns."""
    d = draw(B, T, B, NH, Dk, Dv, "bf16", lens=[T - b for b in range(B)])
    check_forward(S, d, "bf16")
    check_backward(S, d, "bf16")


@pytest.mark.parametrize("dtype,T,B,Dk", [("bf16", 300, 4, 128), ("bf16", 3000, 1, 256), ("bf16", 3000, 1, 64),
                                          ("bf16", 40, 4, 64), ("f32", 3000, 1, 64)])
def test_no_row_has_a_token(S, dtype, T, B, Dk):
    """Every kernel of the call finds nothing to do: zeros, and the states as they came in."""
    d = draw(11, T, B, 2, Dk, Dk, dtype, lens=[0] * B)
    for _ in range(20):
        out = S.linear_attention(d["q"], d["k"], d["v"], d["g"], state=d["s0"], lens=d["lens"], check=False)
        g = S.linear_attention_backward(d["q"], d["k"], d["v"], d["g"], d["do"], state=d["s0"], dstate=d["ds"],
                                        lens=d["lens"], check=False)
        assert torch.equal(out["state"], d["s0"]) and torch.equal(g["dstate"], d["ds"])
        assert not any(t.any() for t in (out["o"], g["dq"], g["dk"], g["dv"]))


def test_state_in_place_across_segments(S):
    """The final state may be written over the initial one."""
    for T in (64, 3000):
        d = draw(5, T, 1, 2, 64, 64, "bf16")
        want = S.linear_attention(d["q"], d["k"], d["v"], d["g"], state=d["s0"])
        from sequential_rnn_gb300._lib import rnn_linattn_desc_t
        desc = rnn_linattn_desc_t(1, T, 1, 2, 64, 64, 0.125, 0)
        s, o = d["s0"].clone(), torch.empty_like(d["v"])
        ws = torch.empty(S.rnn_linattn_workspace_size(desc, 0), dtype=torch.uint8, device="cuda")
        assert S.rnn_linattn_fwd(desc, None, d["q"], d["k"], d["v"], d["g"], None, s, o, s, ws) == 0
        assert S.rnn_read_status(ws) == 0
        assert torch.equal(s, want["state"]) and torch.equal(o, want["o"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_and_broadcast_operands(S, dtype):
    """Views of one fused projection, and keys and values that all heads share."""
    T, B, NH, D = 90, 3, 4, 64
    qkv = draw(6, T, B, 3 * NH, D, D, dtype)["q"]
    d = draw(6, T, B, NH, D, D, dtype)
    d["q"], d["k"], d["v"] = (qkv[:, :, i * NH:(i + 1) * NH] for i in range(3))
    d["do"] = torch.cat([d["do"], d["do"]], -1)[..., :D]
    assert not d["q"].is_contiguous() and not d["do"].is_contiguous()
    plain = {n: x.contiguous() if n in ("q", "k", "v", "do") else x for n, x in d.items()}
    assert torch.equal(check_forward(S, d, dtype)["o"], check_forward(S, plain, dtype)["o"])
    a, b = check_backward(S, d, dtype), check_backward(S, plain, dtype)
    assert all(torch.equal(a[n], b[n]) for n in ("dq", "dk", "dv", "dstate"))
    d["k"], d["v"] = (d[n][:, :, :1].expand(T, B, NH, D) for n in ("k", "v"))
    check_forward(S, d, dtype)
    check_backward(S, d, dtype)   # a gradient for each head; the sharing layer sums them
    one = {n: (x[:1] if n in ("q", "k", "v", "do") else x) for n, x in d.items()}
    check_forward(S, one, dtype)  # a single token of a strided view


def test_offsets_past_32_bits(S):
    """Token strides that put the last tokens over 2^32 bytes and 2^31 elements into the buffer."""
    T, pitch = 600, 4 << 20
    buf = torch.zeros(T * pitch, dtype=torch.bfloat16, device="cuda")
    d = draw(7, T, 1, 2, 64, 64, "bf16")
    for i, n in enumerate(("q", "k", "v")):
        view = buf.as_strided((T, 1, 2, 64), (pitch, 128, 64, 1), 1024 * i)
        view.copy_(d[n])
        d[n] = view
    got = S.linear_attention(d["q"], d["k"], d["v"], d["g"], state=d["s0"])
    d = {n: x.contiguous() if n in ("q", "k", "v") else x for n, x in d.items()}
    want = S.linear_attention(d["q"], d["k"], d["v"], d["g"], state=d["s0"])
    assert torch.equal(got["o"], want["o"]) and torch.equal(got["state"], want["state"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradient_against_differences(S, dtype):
    """The loss is linear in q, in k, in v and in the state: a difference over a whole step is exact,
    up to the forward's own rounding (bounded by its magnitudes)."""
    d = draw(8, 75, 2, 2, 64, 64, dtype, lens=[75, 40])
    got = S.linear_attention_backward(d["q"], d["k"], d["v"], d["g"], d["do"], state=d["s0"], dstate=d["ds"],
                                      lens=d["lens"], scale=0.5)

    def loss(d):
        out = S.linear_attention(d["q"], d["k"], d["v"], d["g"], state=d["s0"], lens=d["lens"], scale=0.5)
        m, f = O.linear_attention_bound(*(np64(d[n]) for n in "qkvg"), np64(d["s0"]), d["lens"].tolist(),
                                        intra=0.5, inter=0.5)
        live = torch.arange(75, device="cuda")[:, None] < d["lens"][None]
        do = d["do"].double() * live[..., None, None]
        # errors are independent from output to output: their root sum of squares, six times
        e = (3 * H if dtype == "bf16" else 2 * U) * np.sqrt(((m[dtype == "f32"] * np64(do.float())) ** 2).sum())
        e += 2 * U * (f * np.abs(np64(d["ds"]))).sum()
        return (out["o"].double() * do).sum().item() + (out["state"].double() * d["ds"].double()).sum().item(), 2 * e

    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("s0", "dstate")):
        step = torch.randn(d[name].shape, device="cuda").to(d[name].dtype)
        hi, lo = ({**d, name: step * s} for s in (2.0, -2.0))   # linear, so around zero as well as anywhere
        if name == "s0":
            hi, lo = {**d, "s0": step * 2}, {**d, "s0": step * -2}
        (a, ea), (b, eb) = loss(hi), loss(lo)
        dot = (got[grad].double() * step.double()).sum().item()
        own = (2 * H if dtype == "bf16" else U) * np.sqrt(((np64(got[grad]) * np64(step)) ** 2).sum()) * 6
        assert abs((a - b) / 4 - dot) <= (ea + eb) / 4 + own + U * abs(dot), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,NH,Dk,Dv", [(1, 1, 32, 32), (5, 3, 64, 64), (2, 6, 128, 128), (3, 2, 256, 256),
                                        (2, 2, 64, 256), (2, 2, 256, 32)])
def test_step(S, B, NH, Dk, Dv, dtype):
    """Tokens one by one: the outputs and the states of the whole sequence."""
    T = 5
    d = draw(9, T, B, NH, Dk, Dv, dtype)
    cache = torch.full((B + 3, NH, Dk, Dv), 7.0, device="cuda")
    slots = torch.randperm(B + 3, device="cuda")[:B].int()
    cache[slots.long()] = d["s0"]
    before = cache.clone()
    got = [S.linear_attention_step(d["q"][t], d["k"][t], d["v"][t], d["g"], cache, slots=slots, scale=0.37)
           for t in range(T)]
    a = [np64(d[n]) for n in ("q", "k", "v", "g")]
    o, s = O.linear_attention(*a, np64(d["s0"]), None, 0.37)
    mag, fin = O.linear_attention_bound(*a, np64(d["s0"]), intra=0.37, inter=0.37)
    tol = (H if dtype == "bf16" else 0) * np.abs(o) + U * mag[1]
    assert (np.abs(np64(torch.stack(got)) - o) <= tol).all()
    close(cache[slots.long()], s, (None, fin), "f32", "state")
    rest = [i for i in range(B + 3) if i not in slots.tolist()]
    assert torch.equal(cache[rest], before[rest])


def test_step_rows_without_a_state_and_strides(S):
    d = draw(10, 1, 4, 3, 64, 64, "bf16")
    cache = d["s0"].clone()
    slots = torch.tensor([2, -1, 4, 0], dtype=torch.int32, device="cuda")
    got = S.linear_attention_step(d["q"][0], d["k"][0], d["v"][0], d["g"], cache, slots=slots)
    assert not got[1].any() and not got[2].any() and torch.equal(cache[[1, 3]], d["s0"][[1, 3]])
    qkv = torch.cat([d["q"][0], d["k"][0], d["v"][0]], 1)
    again = d["s0"].clone()
    same = S.linear_attention_step(*(qkv[:, 3 * i:3 * i + 3] for i in range(3)), d["g"], again, slots=slots)
    assert torch.equal(got, same) and torch.equal(cache, again)
    whole = S.linear_attention_step(d["q"][0], d["k"][0], d["v"][0], d["g"], d["s0"].clone())  # row b: state b
    assert torch.equal(whole[3], S.linear_attention_step(d["q"][0, 3:], d["k"][0, 3:], d["v"][0, 3:], d["g"],
                                                         d["s0"][3:].clone())[0])


def test_empty(S):
    for T, B in ((0, 2), (5, 0)):
        d = draw(11, T, B, 2, 64, 64, "bf16")
        out = S.linear_attention(d["q"], d["k"], d["v"], d["g"], state=d["s0"])
        assert out["o"].shape == (T, B, 2, 64) and torch.equal(out["state"], d["s0"])
        out = S.linear_attention_backward(d["q"], d["k"], d["v"], d["g"], d["do"], dstate=d["ds"])
        assert torch.equal(out["dstate"], d["ds"])


def test_other_stream_and_repeatability(S):
    d = draw(12, 2000, 1, 3, 64, 64, "bf16")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    args = (d["q"], d["k"], d["v"], d["g"])
    want = S.linear_attention(*args, state=d["s0"])
    grad = S.linear_attention_backward(*args, d["do"], state=d["s0"], dstate=d["ds"])
    for handle in (s, s.cuda_stream):
        got = S.linear_attention(*args, state=d["s0"], stream=handle)
        g2 = S.linear_attention_backward(*args, d["do"], state=d["s0"], dstate=d["ds"], stream=handle)
        s.synchronize()
        assert torch.equal(got["o"], want["o"]) and torch.equal(got["state"], want["state"])
        assert all(torch.equal(grad[n], g2[n]) for n in ("dq", "dk", "dv", "dstate"))


def test_graph_capture(S):
    """The calls are launches alone: a captured graph replays on new contents of its inputs."""
    d = draw(13, 1000, 1, 2, 64, 64, "bf16")
    args = (d["q"], d["k"], d["v"], d["g"])
    S.linear_attention(*args, state=d["s0"], check=False)
    S.linear_attention_backward(*args, d["do"], state=d["s0"], dstate=d["ds"], check=False)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = S.linear_attention(*args, state=d["s0"], check=False)
        grad = S.linear_attention_backward(*args, d["do"], state=d["s0"], dstate=d["ds"], check=False)
    d["v"].copy_(draw(14, 1000, 1, 2, 64, 64, "bf16")["v"])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out["o"], S.linear_attention(*args, state=d["s0"])["o"])
    assert torch.equal(grad["dk"], S.linear_attention_backward(*args, d["do"], state=d["s0"], dstate=d["ds"])["dk"])


def test_refusals(S):
    d = draw(15, 8, 2, 2, 64, 64, "bf16")
    args = [d["q"], d["k"], d["v"], d["g"]]
    bad = [(0, d["q"].half(), TypeError), (1, d["k"].float(), TypeError), (1, d["k"][:4], ValueError),
           (2, d["v"][:, :1], ValueError), (3, d["g"][:1], ValueError), (3, d["g"].bfloat16(), TypeError),
           (0, d["q"][0], ValueError), (2, d["v"].cpu(), ValueError),
           (2, d["v"].transpose(0, 3).contiguous().transpose(0, 3), ValueError)]
    for i, t, err in bad:
        with pytest.raises(err):
            S.linear_attention(*[t if j == i else a for j, a in enumerate(args)])
    with pytest.raises(ValueError):
        S.linear_attention(*args, state=d["s0"][:1])
    with pytest.raises(TypeError):
        S.linear_attention(*args, lens=torch.tensor([1, 2], device="cuda"))
    with pytest.raises(ValueError):
        S.linear_attention_backward(*args, d["do"][:4])
    with pytest.raises(ValueError):
        S.linear_attention_step(*(x[0] for x in args[:3]), d["g"], d["s0"][0])
    z = torch.zeros(4, 1, 1, 48, device="cuda")
    with pytest.raises(S.RnnError) as e:
        S.linear_attention(z, z, z, d["g"][:1].clone())
    assert e.value.status == 2
