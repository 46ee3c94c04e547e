"""GPU tests of linear attention with values that are not finite in tokens that count: what they reach, in every
kernel (fp32; mma.sync; tcgen05).

A value at token t reaches what the recurrence hands it to: outputs of t and later tokens of its row and head (in
a gradient's reversed passes, earlier ones), and the state.  Everything else is what it was without it, up to the order of
sums: an output is within 2^-8 (1 + 2^-8) of itself, of its scores' and of its state's magnitudes (bf16; fp32: less) of the
exact one, three times 2^-8 of the sum of magnitudes of all products behind it, and two of them within six
times.  The sum of magnitudes is the operator on absolute values, in fp32.  The states are the same to the bit.
Decays are mild enough that no power of them underflows, which would turn an infinity into NaN.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}

SHAPES = [("f32", 140, 64, 64), ("f32", 100, 256, 32),
          ("bf16", 140, 64, 64), ("bf16", 150, 32, 64), ("bf16", 100, 128, 128), ("bf16", 90, 256, 32),   # mma.sync
          ("bf16", 2000, 64, 64),                                                                     # in segments
          ("bf16", 300, 128, 128), ("bf16", 300, 256, 256), ("bf16", 520, 64, 128), ("bf16", 260, 256, 64),  # tcgen05
          ("bf16", 3000, 128, 128)]                                                                   # in segments


@pytest.fixture(scope="module")
def S():
    from sequential_rnn_gb300 import build
    build.build()
    import sequential_rnn_gb300 as S
    return S


def draw(T, Dk, Dv, dtype):
    B, NH = 3, 2
    g = torch.Generator().manual_seed(T + Dk + Dv)
    f = lambda *s, d="f32", c=1.0: (torch.randn(s, generator=g) * c).to(DT[d]).cuda()  # noqa: E731
    # (from 1 down: not zero, times which an infinity is NaN)
    lens = [T, T - T // 3, 1] if T < 1000 else [T, T // 2, 1]
    return dict(q=f(T, B, NH, Dk, d=dtype), k=f(T, B, NH, Dk, d=dtype, c=Dk ** -0.5), v=f(T, B, NH, Dv, d=dtype),
                g=torch.tensor([-0.02, -0.001]).cuda(), do=f(T, B, NH, Dv, d=dtype), s0=f(B, NH, Dk, Dv),
                ds=f(B, NH, Dk, Dv), lens=torch.tensor(lens, dtype=torch.int32).cuda())


def places(T):
    """Tokens of row 0, and of row 1 whose end is ragged: chunks' first and last tokens and some inside."""
    ends = [t for t in (0, 1, 17, 63, 64, 100, 127, 128, 200, T - 2, T - 1) if t < T]
    return [(t, 0) for t in ends] + [(t, 1) for t in (3, T // 3)]


def forward(S, d):
    out = S.linear_attention(d["q"], d["k"], d["v"], d["g"], state=d["s0"], lens=d["lens"], scale=0.37)
    return {"o": out["o"], "state": out["state"]}


def backward(S, d):
    out = S.linear_attention_backward(d["q"], d["k"], d["v"], d["g"], d["do"], state=d["s0"], dstate=d["ds"],
                                      lens=d["lens"], scale=0.37)
    return {n: out[n] for n in ("dq", "dk", "dv", "dstate")}


# (input, output) -> "column" / "all": later (earlier, for "<") tokens' same column, or all of them; "own": its token alone
REACH = {"v": {"o": ">column", "state": "column", "dq": ">all", "dk": "own"},
         "k": {"o": ">all", "state": "row", "dq": ">column", "dv": "own"},
         "q": {"o": "own", "dk": "<column", "dv": "<all", "dstate": "row"},
         "do": {"dq": "own", "dk": "<all", "dv": "<column", "dstate": "column"}}


def reached(how, out, t, b, h, col):
    m = torch.zeros(out.shape, dtype=torch.bool)
    if how == "row":
        m[b, h, col] = True
    elif how == "column":
        m[b, h, :, col] = True
    else:
        when = {"o": slice(t, t + 1), ">": slice(t, None), "<": slice(0, t + 1)}[how[0]]
        m[when, b, h, col if how.endswith("column") else slice(None)] = True
    return m.cuda()


def behind(out, lens, n):
    """Tokens that do not count."""
    if n in ("state", "dstate"):
        return torch.zeros(out.shape, dtype=torch.bool, device="cuda")
    t = torch.arange(out.shape[0], device="cuda")[:, None] >= lens[None]
    return t[:, :, None, None].expand(out.shape)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype,T,Dk,Dv", SHAPES)
def test_what_a_value_that_is_not_finite_reaches(S, dtype, T, Dk, Dv, value):
    d = draw(T, Dk, Dv, dtype)
    calls = (forward, backward) if T <= 600 or Dk == 128 else (forward,)
    plain = {k: v for f in calls for k, v in f(S, d).items()}
    size = {n: x.float().abs() if n in ("q", "k", "v", "do", "s0", "ds") else x for n, x in d.items()}
    size = {k: v for f in calls for k, v in f(S, size).items()}
    lens = d["lens"].tolist()
    for i, (t, b) in enumerate(places(T)):
        if t >= lens[b]:
            continue
        for name in ("q", "k", "v", "do"):
            h, col = i % 2, (7 * i + 5) % d[name].shape[-1]
            bad = dict(d, **{name: d[name].clone()})
            bad[name][t, b, h, col] = value
            for f in calls:
                for n, out in f(S, bad).items():
                    hit = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
                    if n in REACH[name]:
                        hit = reached(REACH[name][n], out, t, b, h, col) & ~behind(out, d["lens"], n)
                    assert torch.equal(~torch.isfinite(out), hit), (name, n, t, b)
                    rest = torch.where(hit, 0, out.float() - plain[n].float())
                    tol = 0 if n in ("state", "dstate") else 6 * 2.0 ** -8 * (1 + 2.0 ** -7) * size[n]
                    assert (rest.abs() <= tol).all(), (name, n, t, b)


@pytest.mark.parametrize("dtype,T,Dk,Dv", SHAPES)
def test_an_infinity_stays_one_in_the_state(S, dtype, T, Dk, Dv):
    """k_t v_t^T of an infinite k or v is an infinity of the product's sign, and stays one in the state; two of
    opposite sign are NaN.  The same holds for q and do in the initial state's gradient."""
    d = draw(T, Dk, Dv, dtype)
    inf, t0, t1 = float("inf"), T // 2, T // 2 + 2
    for a, c, n in (("k", "v", "state"), ("q", "do", "dstate")):
        if n == "dstate" and T > 600 and Dk != 128:
            continue
        # column 3 of c, row 5 of a: one infinity; column 7 of c, row 9 of a: one of either sign
        x, y = d[a].clone(), d[c].clone()
        y[t0, 0, 0, 3], y[t0, 0, 0, 7], y[t1, 0, 0, 7] = inf, inf, -inf
        x[t0, 0, 1, 5], x[t0, 0, 1, 9], x[t1, 0, 1, 9] = -inf, inf, -inf
        got = (forward if n == "state" else backward)(S, dict(d, **{a: x, c: y}))[n]
        outer = lambda t, h: x[t, 0, h].double()[:, None] * y[t, 0, h].double()[None]  # noqa: E731
        for h, hit in ((0, (slice(None), [3, 7])), (1, ([5, 9], slice(None)))):
            want = (outer(t0, h) + outer(t1, h))[hit]
            assert not want.isfinite().any() and torch.equal(got[0, h][hit].double().nan_to_num(2.0, 1.0, -1.0),
                                                             want.nan_to_num(2.0, 1.0, -1.0)), n
            got[0, h][hit] = 0.0
        assert got.isfinite().all()
