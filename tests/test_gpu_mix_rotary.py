"""GPU tests of the head norm with rotation and its gradient against the fp64 oracle, within the oracle's bounds of fp32
arithmetic (oracle/mix_oracle.py derives them) plus, for bf16 results, half a step of bf16: 2^-8 of the value."""
import numpy as np
import pytest
import torch

from oracle import mix_oracle as O

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = 2.0 ** -126


@pytest.fixture(scope="module")
def S():
    from sequential_rnn_gb300 import build
    build.build()
    import sequential_rnn_gb300 as S
    return S


def np64(t):
    return t.detach().double().cpu().numpy()


def rand(seed, *shape, dtype="f32", scale=1.0):
    x = np.random.default_rng(seed).normal(size=shape) * scale
    return torch.from_numpy(np.asarray(x, np.float32)).to("cuda", DT[dtype])


def close(got, want, err, half=2.0 ** -24):
    got = np64(got)
    tol = err + half * np.abs(want) * (1 + 1e-3) + half * err + TINY
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], tol[bad][:5])


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check(S, q, k, wq, wk, freqs, at, inter, dtype, eps=1e-6):
    dq, dk = (rand(11 + i, *x.shape, dtype=dtype) for i, x in enumerate((q, k)))
    out = dict(zip("qk", S.head_norm_rotary(q, k, wq, wk, freqs, at, eps=eps, interleaved=inter)))
    g = S.head_norm_rotary_backward(q, k, wq, wk, freqs, at, dq, dk, eps=eps, interleaved=inter)
    f, p = None if freqs is None else np64(freqs), None if at is None else at.cpu().numpy()
    four = lambda t: np64(t).reshape((1,) * (4 - t.dim()) + tuple(t.shape))  # noqa: E731
    for n, x, w, d in (("q", q, wq, dq), ("k", k, wk, dk)):
        w64 = None if w is None else np64(w)
        y, err = O.head_norm_rotary(four(x), w64, f, p, eps, inter)
        close(out[n], y.reshape(x.shape), err.reshape(x.shape), HALF[dtype])
        assert out[n].is_contiguous()
        dx, dxe, dw, dwe = O.head_norm_rotary_backward(four(x), w64, f, p, four(d), eps, inter)
        close(g["d" + n], dx.reshape(x.shape), dxe.reshape(x.shape), HALF[dtype])
        if w is None:
            assert "dw" + n not in g
        else:
            close(g["dw" + n], dw, dwe)


# head sizes of every lane count, some with idle lanes, some past the vector kernels'; q and k with different heads
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,B,NQ,NK,D,rot", [
    (1, 1, 1, 1, 2, 2), (3, 2, 3, 1, 6, 4), (5, 3, 2, 2, 8, 8), (1, 16, 12, 12, 64, 64), (4, 5, 3, 3, 32, 32),
    (7, 2, 5, 2, 40, 40), (6, 2, 6, 6, 128, 128), (3, 3, 4, 2, 256, 128), (9, 1, 7, 1, 96, 48), (2, 2, 2, 34, 34, 20),
    (3, 1, 1, 2, 200, 16), (2, 3, 2, 1, 264, 264), (1, 2, 1, 1, 1000, 998), (300, 7, 3, 3, 64, 16), (40, 3, 13, 4, 64, 64)])
def test_shapes(S, T, B, NQ, NK, D, rot, inter, dtype):
    q, k = rand(1, T, B, NQ, D, dtype=dtype, scale=3), rand(2, T, B, NK, D, dtype=dtype)
    wq, wk = 1 + rand(3, D, scale=0.2), 1 + rand(4, D, scale=0.2)
    freqs = S.rotary_frequencies(rot)
    check(S, q, k, wq, wk, freqs, ints(list(range(5, 5 + 1000 * B, 1000))), inter, dtype)


# many tokens: the copies' ring; batches of heads that are full, partial and one head alone
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,B,NQ,NK,D,rot", [
    (350, 7, 13, 1, 64, 64), (2500, 1, 12, 12, 64, 16), (3, 811, 7, 2, 128, 128), (1221, 2, 4, 3, 256, 64), (500, 5, 25, 2, 32, 32)])
def test_many_tokens(S, T, B, NQ, NK, D, rot, inter, dtype):
    qkv = rand(1, T, B, NQ + NK + 1, D, dtype=dtype, scale=2)
    w = 1 + rand(3, 2, D, scale=0.2)
    at = torch.randint(0, 10 ** 6, (B,), generator=torch.Generator().manual_seed(1)).int().cuda()
    check(S, qkv[:, :, :NQ], qkv[:, :, NQ:NQ + NK], w[0], w[1], S.rotary_frequencies(rot), at, inter, dtype)


# the gradient's groups of heads: several of q's, of k's, of both, the last one smaller; fewer tokens than warps
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,B,NQ,NK,D,rot", [
    (410, 3, 33, 13, 128, 128), (1300, 1, 1, 29, 64, 32), (9, 137, 7, 1, 256, 256), (614, 2, 49, 50, 32, 32), (1, 1219, 8, 0, 256, 64)])
def test_head_groups(S, T, B, NQ, NK, D, rot, inter, dtype):
    qkv = rand(1, T, B, NQ + NK, D, dtype=dtype, scale=2)
    w = 1 + rand(3, 2, D, scale=0.2)
    free = torch.randint(-10 ** 6, 10 ** 6, (T, B), generator=torch.Generator().manual_seed(1)).int().cuda()
    check(S, qkv[:, :, :NQ], qkv[:, :, NQ:], w[0], w[1], S.rotary_frequencies(rot), free, inter, dtype)


def test_many_tokens_without_norm_or_rotation(S):
    q, k, w = rand(1, 900, 3, 5, 64, dtype="bf16"), rand(2, 900, 3, 2, 64, dtype="bf16"), 1 + rand(3, 64, scale=0.2)
    f = S.rotary_frequencies(64)
    check(S, q, k, None, None, f, None, False, "bf16")
    check(S, q, k, w, w, None, None, True, "bf16")
    free = torch.randint(-2 ** 31, 2 ** 31 - 1, (900, 3), generator=torch.Generator().manual_seed(1)).int().cuda()
    check(S, q, k, w, w, f, free, False, "bf16")
    check(S, q[:, :, :0], k, w, w, f, free, False, "bf16")


@pytest.mark.parametrize("D", [64, 34])
def test_without_norm_or_rotation(S, D):
    q, k = rand(1, 6, 3, 4, D, dtype="bf16"), rand(2, 6, 3, 4, D, dtype="bf16")
    w, f = 1 + rand(3, D, scale=0.2), S.rotary_frequencies(D)
    check(S, q, k, None, None, f, None, False, "bf16")
    check(S, q, k, w, w, None, None, False, "bf16")
    check(S, q, k, w, w, f[:0], ints([1, 2, 3]), True, "bf16")
    a, b = S.head_norm_rotary(q, k, None, None, None)
    assert torch.equal(a, q) and torch.equal(b, k)


@pytest.mark.parametrize("D", [64, 34])
def test_positions(S, D):
    """Far, negative and free positions; single tokens."""
    T, B = 5, 4
    q, k = rand(1, T, B, 2, D), rand(2, T, B, 2, D)
    w, f = torch.ones(D, device="cuda"), S.rotary_frequencies(D)
    far = ints([0, 2 ** 31 - 1, -2 ** 31, 123456789])
    check(S, q, k, w, w, f, far, False, "f32")
    free = torch.randint(-2 ** 31, 2 ** 31 - 1, (T, B), generator=torch.Generator().manual_seed(1)).int().cuda()
    check(S, q, k, w, w, f, free, True, "f32")
    check(S, q[0], k[0], w, w, f, far, False, "f32")
    # frequencies of more than a turn and of none
    check(S, q, k, w, w, torch.tensor([0.0, 7.5, np.pi, 1e3] * (D // 8), dtype=torch.float64, device="cuda"), far, False, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_views(S, dtype):
    """q, k of one projection; heads in another order; views that begin where no vector may."""
    T, B, NH, D = 6, 3, 4, 64
    w, f, at = 1 + rand(3, D, scale=0.2), S.rotary_frequencies(D), ints([9, 0, 77])
    qkv = rand(1, T, B, 3, NH, D, dtype=dtype)
    q, k, _ = qkv.unbind(2)
    check(S, q, k, w, w, f, at, False, dtype)
    check(S, q.permute(1, 0, 2, 3)[:, :3], k.permute(1, 0, 2, 3)[:, :3], w, w, f, None, True, dtype)
    odd = rand(2, T, B, 2 * NH * D + 1, dtype=dtype)[..., 1:]
    check(S, odd[..., :NH * D].unflatten(-1, (NH, D)), odd[..., NH * D:].unflatten(-1, (NH, D)), w, w, f, at, False, dtype)
    one = rand(4, T, B, 1, D, dtype=dtype)
    check(S, q, one.expand(T, B, 2, D), w, w, f, at, False, dtype)
    # gradients that are views, too
    d = rand(5, T, B, 2, NH, D, dtype=dtype).unbind(2)
    a = S.head_norm_rotary_backward(q, k, w, w, f, at, *d)
    b = S.head_norm_rotary_backward(q, k, w, w, f, at, *[x.contiguous() for x in d])
    for n in a:
        assert torch.equal(a[n], b[n])


def test_zero_heads_and_rows(S):
    w, f = torch.ones(64, device="cuda"), S.rotary_frequencies(64)
    q, k = rand(1, 4, 2, 3, 64), rand(2, 4, 2, 3, 64)
    q[1, 1] = 0  # 0 / sqrt(eps)
    check(S, q, k, w, w, f, ints([0, 5]), False, "f32")
    a, b = S.head_norm_rotary(q, k, w, w, f, eps=0.0)
    assert torch.isnan(a[1, 1]).all() and torch.isfinite(a[0]).all() and torch.isfinite(b).all()
    e = S.head_norm_rotary_backward(q[:, :0], k[:, :0], w, w, f, None, q[:, :0], k[:, :0])
    assert e["dq"].shape == (4, 0, 3, 64) and (e["dwq"] == 0).all() and (e["dwk"] == 0).all()
    a, b = S.head_norm_rotary(q, k[:, :, :0], w, w, f)
    assert torch.equal(a, S.head_norm_rotary(q, k, w, w, f)[0]) and b.numel() == 0


def test_values_that_are_not_finite_stay_in_their_head(S):
    w, f, at = torch.ones(64, device="cuda"), S.rotary_frequencies(64), ints([3, 4])
    q, k = rand(1, 4, 2, 6, 64, dtype="bf16"), rand(2, 4, 2, 3, 64, dtype="bf16")
    bad = q.clone()
    bad[2, 1, 4, 9] = float("inf")
    bad[0, 0, 0, 0] = float("nan")
    a, b = (S.head_norm_rotary(x, k, w, w, f, at) for x in (q, bad))
    hit = torch.zeros(4, 2, 6, dtype=torch.bool, device="cuda")
    hit[2, 1, 4] = hit[0, 0, 0] = True
    assert torch.equal(a[0][~hit], b[0][~hit]) and torch.equal(a[1], b[1]) and torch.isnan(b[0][0, 0, 0]).all()


@pytest.mark.parametrize("T", [4, 1300])  # batches of heads, and the copies' ring
def test_without_norm_the_gradient_does_not_look_at_x(S, T):
    f = S.rotary_frequencies(64)
    q, d = rand(1, T, 2, 3, 64, dtype="bf16"), rand(2, T, 2, 3, 64, dtype="bf16")
    bad = torch.full_like(q, float("nan"))
    bad[::2] = float("inf")
    a, b = (S.head_norm_rotary_backward(x, x, None, None, f, None, d, d) for x in (q, bad))
    assert torch.equal(a["dq"], b["dq"]) and torch.equal(a["dk"], b["dk"]) and torch.isfinite(b["dq"]).all()


def test_captured_and_repeated(S):
    T, B, NH, D = 50, 4, 6, 128
    q, k, dq, dk = (rand(i, T, B, NH, D, dtype="bf16") for i in range(4))
    w, f, at = 1 + rand(9, D, scale=0.1), S.rotary_frequencies(D), ints([1, 2, 3, 4])

    def run():
        g = S.head_norm_rotary_backward(q, k, w, w, f, at, dq, dk)
        return [*S.head_norm_rotary(q, k, w, w, f, at), *g.values()]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for i, x in enumerate((q, k, dq, dk)):
        x.copy_(rand(20 + i, T, B, NH, D, dtype="bf16"))
    at += 1000
    for _ in range(2):
        graph.replay()
        for a, b in zip(got, run()):
            assert torch.equal(a, b)


def test_refusals(S):
    q, w, f = rand(1, 4, 2, 3, 64), torch.ones(64, device="cuda"), S.rotary_frequencies(64)
    for a, kw, e in (((q, q, w, None, f), {}, ValueError), ((q, q, w, w[:32], f), {}, ValueError),
                     ((q, q.bfloat16(), w, w, f), {}, TypeError), ((q, q[:3], w, w, f), {}, ValueError),
                     ((q, q, w, w, f.float()), {}, TypeError), ((q, q, w, w, torch.cat([f, f])), {}, ValueError),
                     ((q, q, w, w, f, ints([1])), {}, ValueError), ((q, q, w, w, f, ints([[1, 2]])), {}, ValueError),
                     ((q, q, w, w, f, ints([1, 2]).long()), {}, TypeError), ((q, q[0], w, w, f), {}, ValueError),
                     ((q[0, 0], q[0, 0], w, w, f), {}, ValueError), ((q.half(), q.half(), w, w, f), {}, TypeError),
                     ((q.transpose(2, 3), q.transpose(2, 3), w[:3], w[:3], None), {}, ValueError),
                     ((q, q, w, w, f), dict(eps=-1.0), S.RnnError)):
        with pytest.raises(e):
            S.head_norm_rotary(*a, **kw)
    odd = rand(1, 2, 2, 2, 7)
    with pytest.raises(S.RnnError):
        S.head_norm_rotary(odd, odd, None, None, None)
    with pytest.raises(ValueError):
        S.head_norm_rotary_backward(q, q, w, w, f, None, q[:, :, :2], q)
