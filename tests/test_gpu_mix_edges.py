"""GPU tests of the gated recurrence, the head norm with rotation and the clipping where a lost term or a value that is not
finite would pass the operators' other tests.  Tolerances as there (the oracle's bounds), or exact."""
import numpy as np
import pytest
import torch

from oracle import mix_oracle as O
from tests.test_gpu_mix_rotary import DT, S, check, close, ints, np64, rand  # noqa: F401 (S: the fixture)

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


# ------------------------------------------------------------------ rotation --
# heads that fill no whole batch of lanes; vector forms of both pair layouts, value by value, the ring, heads above 256
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H", [1, 3, 5])
@pytest.mark.parametrize("T,B,D,rot,inter", [
    (5, 3, 32, 32, False), (5, 3, 64, 64, False), (4, 3, 128, 64, True), (6, 2, 34, 20, False), (5, 3, 100, 98, True),
    (5, 2, 264, 128, False), (613, 2, 64, 64, False), (613, 2, 128, 128, True)])
def test_gradient_without_eps(S, T, B, H, D, rot, inter, dtype):
    q, k = rand(1, T, B, H, D, dtype=dtype, scale=3), rand(2, T, B, 1 + H % 3, D, dtype=dtype)
    w = 1 + rand(3, 2, D, scale=0.2)
    check(S, q, k, w[0], w[1], S.rotary_frequencies(rot), ints(list(range(7, 7 + B))), inter, dtype, eps=0.0)


@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("D", [264, 1000, 34, 128])
def test_without_norm_the_gradient_does_not_look_at_x(S, D, T):
    f = S.rotary_frequencies(D // 4 * 2)
    q, d = rand(1, T, 2, 3, D, dtype="bf16"), rand(2, T, 2, 3, D, dtype="bf16")
    bad = torch.full_like(q, NAN)
    bad[::2] = INF
    a, b = (S.head_norm_rotary_backward(x, x, None, None, f, None, d, d) for x in (q, bad))
    assert torch.equal(a["dq"], b["dq"]) and torch.equal(a["dk"], b["dk"]) and torch.isfinite(b["dq"]).all()


# batches of heads (pieces of four, pairs of which some of a lane's turn, value by value), the rings, heads above 256
PART = [(9, 2, 3, 64, 16, False), (9, 2, 3, 64, 12, True), (9, 2, 3, 64, 20, False), (9, 2, 3, 34, 20, True), (4, 2, 7, 256, 128, False),
        (700, 2, 3, 64, 16, False), (700, 2, 3, 64, 12, True), (700, 2, 2, 128, 0, False), (9, 1, 2, 128, 0, True),
        (40, 2, 3, 264, 64, False), (40, 2, 3, 264, 64, True)]


def spoilt(x, rot, value):
    """x with `value` in one column from rot on of every other head, another one in each; and where."""
    D = x.shape[-1]
    bad, at = x.clone(), torch.zeros(x.shape, dtype=torch.bool, device="cuda")
    rows = torch.arange(0, x.numel() // D, 2, device="cuda")
    cols = rot + (rows // 2) % (D - rot)
    bad.view(-1, D)[rows, cols] = value
    at.view(-1, D)[rows, cols] = True
    return bad, at


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [INF, -INF, NAN])
@pytest.mark.parametrize("T,B,H,D,rot,inter", PART)
def test_columns_that_do_not_turn_stay_apart(S, T, B, H, D, rot, inter, value, dtype):
    """What is not finite in a column past the rotation reaches no other column, without a norm; of the weights' gradients only
    its own."""
    x, f = rand(1, T, B, H, D, dtype=dtype), S.rotary_frequencies(rot)
    bad, at = spoilt(x, rot, value)
    for call in (lambda v: S.head_norm_rotary(v, v, None, None, f, interleaved=inter),
                 lambda v: tuple(S.head_norm_rotary_backward(x, x, None, None, f, None, v, v, interleaved=inter).values())):
        a, b = call(x), call(bad)
        for y, z in zip(a, b):
            assert torch.equal(y[~at], z[~at])
            assert torch.isnan(z[at]).all() if value != value else (z[at] == value).all()
    w = 1 + rand(3, D, scale=0.2)
    one = torch.zeros_like(at)
    one.view(-1, D)[0] = at.view(-1, D)[0]
    d = torch.where(one, bad, x)
    a, b = (S.head_norm_rotary_backward(x, x, w, w, f, None, v, v, interleaved=inter) for v in (x, d))
    for n in ("dwq", "dwk"):
        keep = torch.arange(D, device="cuda") != rot
        assert torch.equal(a[n][keep], b[n][keep]) and not torch.isfinite(b[n][rot])


@pytest.mark.parametrize("T,B,H,D,rot,inter", PART)
def test_an_infinity_leaves_zeros_in_columns_that_do_not_turn(S, T, B, H, D, rot, inter):
    """1 / sqrt(mean x^2) of its head is zero, and so is every finite value's product with it."""
    x, w = rand(1, T, B, H, D), torch.ones(D, device="cuda")
    bad, at = spoilt(x, rot, INF)
    y = S.head_norm_rotary(bad, bad, w, w, S.rotary_frequencies(rot), interleaved=inter)[0]
    hit = at.any(-1, keepdim=True).expand_as(at).clone()
    assert torch.isnan(y[at]).all() and (y[hit & ~at] == 0).all()


# shapes of every kernel: batches (lanes that idle, value by value), rings with one group and with several, heads above 256
TERMS = [(5, 3, 5, 3, 64), (100, 3, 13, 1, 32), (700, 1, 3, 2, 40), (600, 3, 7, 5, 34), (1300, 1, 5, 3, 96), (350, 7, 13, 1, 64),
         (3, 811, 7, 2, 128), (500, 5, 25, 2, 32), (410, 3, 33, 13, 128), (1300, 1, 1, 29, 64), (9, 137, 7, 1, 256),
         (614, 2, 49, 50, 32), (1, 1219, 8, 0, 256), (50, 13, 3, 2, 264)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,B,NQ,NK,D", TERMS)
def test_no_term_of_a_weight_gradient_is_lost(S, T, B, NQ, NK, D, dtype):
    """With x = dy = 1, eps = 3 and no rotation every term is 1 / sqrt(4): the sum is half their number.  Its error is
    that of the root (2^-22 of it) and one rounding for each sum on a term's way, of which there are less than 100 (terms of a
    lane, lanes, warps, CTAs): below a quarter, half a term."""
    x = [torch.ones(T, B, n, D, dtype=DT[dtype], device="cuda") for n in (NQ, NK)]
    w = 1 + rand(3, 2, D, scale=0.2)
    g = S.head_norm_rotary_backward(*x, w[0], w[1], None, None, *x, eps=3.0)
    for n, H in (("dwq", NQ), ("dwk", NK)):
        assert T * B * H / 2 * (4 + 100) * 2.0 ** -24 < 0.25
        assert ((g[n] - T * B * H / 2).abs() < 0.25).all(), (n, g[n])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,B,NQ,NK,D", TERMS)
def test_a_weight_gradient_of_one_head(S, T, B, NQ, NK, D, dtype):
    """dy in one head of one token alone, at the ends of tokens and of heads."""
    q, k = rand(1, T, B, NQ, D, dtype=dtype), rand(2, T, B, NK, D, dtype=dtype)
    w, f = 1 + rand(3, 2, D, scale=0.2), S.rotary_frequencies(D // 2 * 2)
    dy = rand(4, 1, 1, 1, D, dtype=dtype)
    for t, b, h in ((0, 0, 0), (T - 1, B - 1, -1), (T // 2, 0, -1), (T - 1, 0, 0), (0, B - 1, -2), (T // 3, B // 2, 3)):
        d = [torch.zeros_like(x) for x in (q, k)]
        for x in d:
            if x.shape[2]:
                x[t, b, h % x.shape[2]] = dy
        g = S.head_norm_rotary_backward(q, k, w[0], w[1], f, None, *d)
        for i, (n, x) in enumerate((("q", q), ("k", k))):
            if x.shape[2] == 0:
                assert (g["dw" + n] == 0).all()
                continue
            one = x[t:t + 1, b:b + 1, h % x.shape[2]][:, :, None]
            _, _, dw, dwe = O.head_norm_rotary_backward(np64(one), np64(w[i]), np64(f), np.array([[t]]), np64(dy), 1e-6, False)
            close(g["dw" + n], dw, dwe)
            hit = torch.zeros_like(x, dtype=torch.bool)
            hit[t, b, h % x.shape[2]] = True
            assert (g["d" + n][~hit] == 0).all()


def test_a_weight_gradient_of_a_late_head(S):
    """dy in one head behind 2^31 values, in the last token of a row and in one before it."""
    if torch.cuda.get_device_properties(0).total_memory < 60 << 30:
        pytest.skip("needs 60 GB")
    T, B, NH, D = 4100, 64, 64, 128
    q = torch.randn(T, B, NH, D, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda", dtype=torch.bfloat16)
    k, w, f = q[:, :, :2], 1 + rand(3, D, scale=0.2), S.rotary_frequencies(D)
    d, dy = torch.zeros_like(q), rand(4, 1, 1, 1, D, dtype="bf16")
    for t, b, h in ((T - 1, B - 1, NH - 1), (T - 2, 0, 1)):
        d[t, b, h] = dy
        g = S.head_norm_rotary_backward(q, k, w, w, f, None, d, d[:, :, :2])
        _, _, dw, dwe = O.head_norm_rotary_backward(np64(q[t:t + 1, b:b + 1, h:h + 1]), np64(w), np64(f), np.array([[t]]), np64(dy),
                                                    1e-6, False)
        close(g["dwq"], dw, dwe)
        close(g["dwk"], dw * (h < 2), dwe)
        d[t, b, h] = 0
        del g


# ------------------------------------------------------------------ clipping --
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_value_of_a_norm_is_lost(S, dtype):
    """One value that is not zero, at the ends of vectors, units, tensors and launches' tables: exact norms and factors."""
    size = [5_000_001, 1, 8192, 4097] + [3 + i % 5 for i in range(300)]
    flat = [torch.zeros(n, dtype=DT[dtype], device="cuda") for n in size]
    unit = 16384 // flat[0].element_size()
    at = [(0, i) for i in (0, 7, 8, unit - 1, unit, 300 * unit - 1, 300 * unit, size[0] // unit * unit, size[0] - 2, size[0] - 1)]
    at += [(i, n - 1) for i, n in ((1, 1), (2, 8192), (3, 4097), (15, size[15]), (255, size[255]), (256, size[256]), (303, size[303]))]
    for i, j in at:
        flat[i][j] = -3.0
        assert S.grad_norm(flat).item() == 3.0
        assert S.clip_grad_norm(flat, 0.75).item() == 3.0
        assert flat[i][j].item() == -0.75 and S.grad_norm(flat).item() == 0.75, (i, j)
        flat[i][j] = 0.0


def test_no_value_of_a_long_tensor_is_lost(S):
    n = 2 ** 31 + 4099
    if torch.cuda.get_device_properties(0).total_memory < 20 << 30:
        pytest.skip("needs 20 GB")
    x = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    for j in (0, 2 ** 31 - 1, 2 ** 31, n - 1):
        x[j] = 3.0
        assert S.clip_grad_norm([x], 1.5).item() == 3.0 and x[j].item() == 1.5
        x[j] = 0.0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [33, 4096, 100003, 3_000_001, 60_000_000])
def test_norm_of_many_values(S, n, dtype):
    """A thread's 64 bytes (32 bf16 values) are summed in four chains of at most 8 in fp32, then in two sums: 10
    roundings; above them sums carry their rounding errors along, and a CTA's are fp64.  Half of that in the root, and its
    own rounding: 6 2^-24 (7, with what the carried errors lose)."""
    x = torch.randn(n, generator=torch.Generator(device="cuda").manual_seed(n), device="cuda", dtype=DT[dtype])
    want = np.sqrt(sum(float(c.double().square().sum()) for c in x.split(1 << 24)))
    assert abs(S.grad_norm([x]).item() - want) <= 7 * 2.0 ** -24 * want


# ------------------------------------------------------- gated recurrence --
def config(S, T, B, NH, D, gates, dtype, gradient=False):
    from sequential_rnn_gb300._lib import GATE_COUNTS, rnn_gated_desc_t
    return S.rnn_gated_config(rnn_gated_desc_t(int(dtype == "bf16"), T, B, NH, D, GATE_COUNTS[gates], 0), gradient)


@pytest.mark.parametrize("gradient", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,B,NH,D,gates", [
    (16384, 1, 12, 32, "fz"), (16384, 1, 3, 128, "fz"), (16384, 1, 12, 64, "fz"), (16384, 1, 8, 64, "fzo"), (8000, 2, 6, 64, "fz"),
    (8192, 1, 10, 64, "fzo"), (4000, 4, 4, 64, "fz"), (1000, 5, 3, 64, "fz"), (500, 8, 2, 64, "fz"), (16384, 1, 3, 32, "ifzo")])
def test_planned_clusters_are_there_at_once(S, T, B, NH, D, gates, dtype, gradient):
    """The plan counts on it at these sizes: no cluster waits for another one to leave, whatever shared memory spreads them."""
    c = config(S, T, B, NH, D, gates, dtype, gradient)
    assert c["tile"] and c["grid"] % c["cluster"] == 0 and c["held"] >= c["grid"] // c["cluster"], c


# (channels of a tile, maps a round ahead, CTAs of a cluster: 1, up to 8, more)
@pytest.mark.parametrize("dtype,gradient,T,B,NH,D,kernel", [
    ("bf16", False, 65, 40, 5, 40, (32, 0, 1)), ("bf16", False, 1000, 40, 1, 8, (32, 0, 8)), ("bf16", False, 1500, 30, 1, 8, (32, 0, 16)),
    ("bf16", False, 65, 8, 12, 32, (32, 1, 1)), ("bf16", False, 200, 40, 1, 8, (32, 1, 8)), ("bf16", False, 1500, 1, 1, 8, (32, 1, 16)),
    ("bf16", False, 129, 40, 4, 72, (64, 0, 1)), ("bf16", False, 129, 16, 4, 72, (64, 0, 8)), ("bf16", False, 600, 16, 2, 40, (64, 0, 16)),
    ("bf16", False, 129, 30, 5, 40, (64, 1, 1)), ("bf16", False, 65, 1, 1, 8, (64, 1, 8)), ("bf16", False, 600, 1, 1, 8, (64, 1, 16)),
    ("bf16", True, 65, 1, 1, 8, (32, 0, 1)), ("bf16", True, 200, 40, 1, 8, (32, 0, 8)), ("bf16", True, 1500, 1, 1, 8, (32, 0, 16)),
    ("bf16", True, 129, 16, 4, 72, (64, 0, 1)), ("bf16", True, 129, 1, 1, 8, (64, 0, 8)), ("bf16", True, 600, 1, 1, 8, (64, 0, 16)),
    *[("f32", g, *size) for g in (False, True) for size in
      ((65, 40, 5, 40, (32, 0, 1)), (100, 40, 1, 8, (32, 0, 8)), (600, 1, 1, 8, (32, 0, 16)), (65, 30, 5, 40, (64, 0, 1)),
       (65, 1, 1, 8, (64, 0, 8)), (257, 1, 1, 8, (64, 0, 16)))],
    ("bf16", False, 65, 3, 2, 33, (0, 0, 8)), ("f32", True, 64, 3, 2, 32, (0, 0, 1))])
def test_every_planned_kernel(S, dtype, gradient, T, B, NH, D, kernel):
    """Against the oracle, at sizes that take it (of the device that the plan's rounds were measured on)."""
    from tests.test_gpu_mix_gated import check as check_gated
    c = config(S, T, B, NH, D, "fz", dtype, gradient)
    cluster = next(n for n in (1, 8, 16) if c["cluster"] <= n)
    assert (c["tile"], c["ahead"], cluster) == kernel, c
    check_gated(S, T, B, NH, D, "fz", dtype, seed=T + D)
    check_gated(S, T, B, NH, D, "fz", dtype, lens=[T - (b * 37) % (T + 1) for b in range(B)], seed=T)


def test_the_timeout_flag_is_refused_where_no_tile_is_brought(S):
    """Addresses that have no tensor map run on kernels that wait for nothing."""
    from sequential_rnn_gb300._lib import RNN_FLAG_TEST_TIMEOUT, rnn_gated_desc_t
    T, B, NH, D = 100, 2, 1, 32
    d = rnn_gated_desc_t(1, T, B, NH, D, 2, RNN_FLAG_TEST_TIMEOUT)
    Wx = torch.zeros(T * B * NH * 2 * D + 1, dtype=torch.bfloat16, device="cuda")[1:]
    y = torch.zeros(T * B * NH * D, dtype=torch.bfloat16, device="cuda")
    stash = torch.zeros(13 * B * NH * D, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    assert S.rnn_gated_fwd(d, Wx, None, None, y, None, None, ws) == 2
    assert S.rnn_gated_bwd(d, Wx, None, stash, y, None, torch.empty_like(Wx), None, ws) == 2


# ------------------------------------------------------ what is written in place --
def test_what_is_written_in_place_counts_as_changed(S):
    """Automatic differentiation that saved such a tensor notices; the norm alone writes nothing."""
    x, none = rand(1, 64), torch.empty(0, device="cuda")
    leaf = rand(2, 64).requires_grad_()
    y = (leaf * x).sum()
    at = x._version
    S.grad_norm([x])
    assert x._version == at
    S.clip_grad_norm([x, none], 1e-3)
    assert x._version > at
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    state, Wx = rand(3, 4, 2, 8), rand(4, 4, 2, 16)
    at = state._version
    S.gated_recurrence_step(Wx, state)
    assert state._version > at
    q, memory = rand(6, 4, 2, 64), rand(7, 4, 2, 64, 64)
    at = memory._version
    S.linear_attention_step(q, q, q, torch.zeros(2, device="cuda"), memory)
    assert memory._version > at
    with torch.inference_mode():  # such tensors have no version
        z = rand(5, 64)
        S.clip_grad_norm([z], 1e-3)
        S.gated_recurrence_step(Wx, state.clone())
    S.clip_grad_norm([z], 1e-4)


# ------------------------------------------------------------------- example --
def test_a_rotary_layers_positions_are_its_live_tokens(S):
    """Lengths beyond the prompt and below zero are taken as its length and none."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import linear_attention_lm as ex
    m = ex.Model(2, 64, layers=("rotary",), seed=5)
    x = rand(1, 20, 3, 128, dtype="bf16")
    _, a = m.prompt(x, ints([20, 0, 7]))
    _, b = m.prompt(x, ints([25, -4, 7]))
    assert torch.equal(a[0][0], b[0][0]) and torch.equal(a[0][1], b[0][1]) and a[0][1].tolist() == [20, 0, 7]
