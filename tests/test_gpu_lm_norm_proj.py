"""GPU tests of the root-mean-square norm (bf16, fp32 and 8-bit outputs, gradient), the
weight quantiser and the 8-bit projection, against the fp64 oracle.

Tolerances, from the number formats:
 - a bf16 result is the fp32 one rounded once: 2^-8 of it (half of the spacing of 8-bit
   significands), plus fp32 sum error;
 - fp32 sums of up to 16392 terms: 2^-18 of the sum of magnitudes;
 - an e4m3 value is half a step off (2^-4 of it, 2^-10 of the scale when subnormal) from y / scale, and
   the scale 2^-20 of itself; a value whose y / scale lies within the fp32 error of the
   middle of two steps may take either.
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import lm_oracle as O

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -18


@pytest.fixture(scope="module")
def S():
    from sequential_rnn_gb300 import build
    build.build()
    import sequential_rnn_gb300 as S
    return S


def rand(seed, *shape, dtype="f32", scale=1.0):
    x = np.random.default_rng(seed).normal(size=shape).astype(np.float32) * scale
    return torch.from_numpy(np.asarray(x, np.float32)).to("cuda", DT[dtype])


def np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


SHAPES = [(1, 1), (3, 7), (2, 8), (5, 100), (4, 127), (4, 128), (3, 129), (17, 768), (33, 1000), (9, 1001),
          (300, 256), (5, 4096), (3, 8200), (2, 16392), (2, 16385)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,N", SHAPES)
def test_rms_norm(S, rows, N, dtype):
    x, res, w = rand(1, rows, N, dtype=dtype), rand(2, rows, N, dtype=dtype, scale=3), rand(3, N)
    out = S.rms_norm(x, w, res, eps=1e-5, train=True)
    h = (x.float() + res.float()).to(DT[dtype])
    assert torch.equal(out["h"], h)
    y, r = O.rms_norm(np64(h), np64(w), 1e-5)
    step = 2.0 ** -8 if dtype == "bf16" else 0.0
    assert (np.abs(np64(out["y"]) - y) <= (step + U) * np.abs(y)).all()
    np.testing.assert_allclose(np64(out["rstd"]), r, rtol=U)
    alone = S.rms_norm(h, w, eps=1e-5)
    assert alone["h"] is h and torch.equal(alone["y"], out["y"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,N", SHAPES)
def test_rms_norm_8bit(S, rows, N, dtype):
    x, res, w = rand(4, rows, N, dtype=dtype), rand(5, rows, N, dtype=dtype), rand(6, N)
    x[0, :min(N, 128)] = -res[0, :min(N, 128)]   # a block of zeros
    out = S.rms_norm(x, w, res, quantize=True)
    h = (x.float() + res.float()).to(DT[dtype])
    assert torch.equal(out["h"], h)
    y, _ = O.rms_norm(np64(h), np64(w), 1e-6)
    q, s = O.quantize(y)
    np.testing.assert_allclose(np64(out["scale"]), s, rtol=2.0 ** -20 + U)
    full = np.repeat(s, 128, 1)[:, :N]
    tol = (2.0 ** -4 + U) * np.abs(y) + full * 2.0 ** -10
    assert (np.abs(np64(out["y"]) * full - y) <= tol).all()
    assert (np64(out["y"]) != q).mean() <= 1e-3 + (2.0 if q.size < 100 else 0)
    assert out["scale"][0, 0] == 1 and not np64(out["y"])[0, :min(N, 128)].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("small", [1.0, 2.0 ** -114, 2.0 ** -128, 2.0 ** -135, "ones", "short"])
@pytest.mark.parametrize("rows,N", [(2000, 768), (700, 1001), (40, 8192), (5, 16512)])
def test_rms_norm_8bit_codes_are_the_nearest(S, rows, N, small, dtype):
    """y / scale = 448 h w / max|h w|, of which 64 bits hold the products exactly, rounded to fp32 and then to 8
    bits: equal codes, at every magnitude a scale can have (by a subnormal one, which is coarse, the quotient is that of
    what is stored)."""
    x, w = rand(60, rows, N, dtype=dtype), rand(61, N, scale=small if isinstance(small, float) else 1.0)
    if small == "ones":                           # products of 8 bits: many exact ties
        w = torch.ones_like(w)
    if small == "short":
        x, w, small = x.bfloat16().to(x.dtype), w.bfloat16().float(), 1.0
    small = 1.0 if small == "ones" else small
    out = S.rms_norm(x, w, quantize=True, train=True)
    hw, s = np64(x) * np64(w), np.repeat(np64(out["scale"]), 128, 1)[:, :N]
    pad = np.pad(np.abs(hw), ((0, 0), (0, -N % 128))).reshape(rows, -1, 128).max(2)
    q = np.where(s >= 2.0 ** -126, 448 * hw / np.repeat(pad, 128, 1)[:, :N], hw * (np64(out["rstd"])[:, None] / s))
    assert (s < 2.0 ** -126).any() == (small < 2.0 ** -120)
    assert np.array_equal(np64(out["y"]), O.e4m3(q.astype(np.float32)))


def test_rms_norm_leading_dimensions_in_place_and_empty(S):
    x, res, w = rand(7, 3, 5, 256, dtype="bf16"), rand(8, 3, 5, 256, dtype="bf16"), rand(9, 256)
    want = S.rms_norm(x, w, res, quantize=True, train=True)
    assert want["scale"].shape == (3, 5, 2) and want["rstd"].shape == (3, 5)
    for over in ("x", "residual"):                # h in the place of either input
        a, b = x.clone(), res.clone()
        y, h = torch.empty_like(x), a if over == "x" else b
        st = S.rnn_rms_norm(1, 15, 256, 1e-6, a, b, w, h, y, None, None)
        assert st == 0 and torch.equal(h, want["h"])
        assert torch.equal(y, S.rms_norm(x, w, res)["y"])
    none = S.rms_norm(x[:0], w, res[:0], quantize=True)
    assert none["y"].shape == (0, 5, 256) and none["scale"].shape == (0, 5, 2)


def test_rms_norm_values_that_are_not_finite(S):
    x, w = rand(10, 4, 256), rand(11, 256)
    x[1, 3], x[2, 200] = float("nan"), float("inf")
    for quantize in (False, True):
        out = S.rms_norm(x, w, quantize=quantize)
        y = out["y"].float()
        clean = S.rms_norm(x[[0, 3]], w, quantize=quantize)["y"].float()
        assert torch.equal(y[[0, 3]], clean)      # other rows do not notice
        assert y[1].isnan().all() and y[2].isnan().any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,N", SHAPES + [(2000, 96), (1300, 1000)])
def test_rms_norm_backward(S, rows, N, dtype):
    h, dy, dh, w = (rand(20, rows, N, dtype=dtype, scale=2), rand(21, rows, N, dtype=dtype),
                    rand(22, rows, N, dtype=dtype), rand(23, N))
    _, r = O.rms_norm(np64(h), np64(w), 1e-6)
    rstd = torch.from_numpy(r.astype(np.float32)).cuda()
    step = 2.0 ** -8 if dtype == "bf16" else 0.0
    for extra in (dh, None):
        got = S.rms_norm_backward(dy, h, w, rstd, dh=extra)
        dx, dw = O.rms_norm_backward(np64(dy), np64(h), np64(w), np64(rstd), None if extra is None else np64(extra))
        g, xh = np64(dy) * np64(w), np64(h) * np64(rstd)[:, None]
        mag = np64(rstd)[:, None] * (np.abs(g) + np.abs(xh) * np.abs(g * xh).mean(1, keepdims=True))
        mag = mag + (0 if extra is None else np.abs(np64(extra)))
        assert (np.abs(np64(got["dx"]) - dx) <= step * np.abs(dx) + 4 * U * mag).all()
        assert (np.abs(np64(got["dw"]) - dw) <= U * np.abs(np64(dy) * xh).sum(0)).all()
        again = S.rms_norm_backward(dy, h, w, rstd, dh=extra)
        assert torch.equal(got["dw"], again["dw"]) and torch.equal(got["dx"], again["dx"])


def test_rms_norm_backward_against_differences(S):
    """f32: the loss sum(y dy) along a direction, central differences in fp64 of the kernel's y."""
    h, dy, w = rand(24, 6, 192), rand(25, 6, 192), rand(26, 192)
    d = rand(27, 6, 192)
    out = S.rms_norm(h, w, train=True)
    got = S.rms_norm_backward(dy, h, w, out["rstd"])
    e = 2.0 ** -6
    f = lambda h: (S.rms_norm(h, w)["y"].double() * dy.double()).sum().item()  # noqa: E731
    # truncation e^2 / 6 of the third derivative (of order the loss's magnitude), rounding 2^-22 / e of it
    mag = (dy.double().abs() * out["y"].double().abs()).sum().item()
    assert abs((f(h + e * d) - f(h - e * d)) / (2 * e) - (got["dx"].double() * d.double()).sum().item()) <= \
        (e * e + 2.0 ** -22 / e) * mag
    f = lambda w: (S.rms_norm(h, w)["y"].double() * dy.double()).sum().item()  # noqa: E731
    dw = rand(28, 192)
    assert abs((f(w + dw) - f(w - dw)) / 2 - (got["dw"].double() * dw.double()).sum().item()) <= 2.0 ** -16 * mag * 4


def test_rms_norm_backward_no_rows(S):
    z = torch.zeros(0, 64, device="cuda")
    got = S.rms_norm_backward(z, z, rand(1, 64), torch.zeros(0, device="cuda"))
    assert got["dx"].shape == (0, 64) and not got["dw"].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,K", [(1, 1), (128, 128), (130, 300), (257, 129), (768, 784)])
def test_quantize_weight(S, N, K, dtype):
    W = rand(30, N, K, dtype=dtype)
    W[:min(N, 128), :min(K, 128)] *= 0 if N > 200 else 1
    Wq, Ws = S.quantize_weight(W)
    q, s = O.quantize(np64(W), 128)
    np.testing.assert_allclose(np64(Ws), s, rtol=2.0 ** -22)
    full = np.repeat(np.repeat(s, 128, 0)[:N], 128, 1)[:, :K]
    assert (np.abs(np64(Wq) * full - np64(W)) <= (2.0 ** -4 + U) * np.abs(np64(W)) + full * 2.0 ** -10).all()
    assert (np64(Wq) != q).mean() <= 1e-3 + (2.0 if q.size < 100 else 0)


def operands(M, N, K, seed):
    r = np.random.default_rng(seed)
    x, w = r.normal(size=(M, K)), r.normal(size=(N, K)) / np.sqrt(K)
    x[:, :1] *= 30
    xq, xs = O.quantize(x)
    wq, ws = O.quantize(w, 128)
    b = r.normal(size=N).astype(np.float32)
    t = lambda a, d: torch.from_numpy(a.astype(np.float32)).to("cuda", d)  # noqa: E731
    e4 = torch.float8_e4m3fn
    xs, ws = xs.astype(np.float32), ws.astype(np.float32)
    return (t(xq, e4), t(xs, torch.float32), t(wq, e4), t(ws, torch.float32), t(b, torch.float32)), \
        O.proj_fp8(xq, xs, wq, ws, b)


@pytest.mark.parametrize("M,N,K", [
    (1, 8, 16), (1, 2304, 768), (3, 136, 144), (8, 768, 1024), (16, 2304, 768), (17, 264, 400), (32, 4096, 256),
    (33, 512, 2048), (64, 128, 128), (65, 1000, 784), (127, 128, 1040), (128, 256, 128), (129, 120, 4096),
    (257, 2312, 784), (1000, 768, 768), (1024, 2304, 256), (2049, 1032, 1024), (5000, 264, 16), (4096, 4096, 272)])
def test_input_proj_fp8(S, M, N, K):
    (xq, xs, wq, ws, b), (want, mag) = operands(M, N, K, M + N + K)
    got = np64(S.input_proj_fp8(xq, xs, wq, ws, b))
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + U * mag).all()
    got = np64(S.input_proj_fp8(xq.view(1, M, K), xs.view(1, M, -1), wq, ws))[0]
    want = want - np64(b)
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + U * mag).all()


@pytest.mark.parametrize("M,N,K", [(16, 4872, 272), (17, 4864, 144), (17, 4872, 144), (40, 4872, 272), (64, 6000, 128),
                                   (33, 2432, 144), (33, 2440, 400), (16, 9728, 144), (1, 9736, 144), (9, 9736, 272)])
def test_input_proj_fp8_few_rows_of_many_columns(S, M, N, K):
    """Both sides of the places where another kernel takes over."""
    (xq, xs, wq, ws, b), (want, mag) = operands(M, N, K, M + N + K)
    got = np64(S.input_proj_fp8(xq, xs, wq, ws, b))
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + U * mag).all()


def test_input_proj_fp8_row_isolation_and_no_rows(S):
    """A row of NaN stays in its row; nothing is done for no rows."""
    (xq, xs, wq, ws, b), _ = operands(130, 200, 384, 5)
    clean = S.input_proj_fp8(xq, xs, wq, ws, b)
    for rows in (130, 12):                        # either kernel
        bad = xs[:rows].clone()
        bad[7] = float("nan")
        got = S.input_proj_fp8(xq[:rows].contiguous(), bad, wq, ws, b)
        keep = [i for i in range(rows) if i != 7]
        assert got[7].isnan().all() and not got[keep].isnan().any()
        if rows == 130:
            assert torch.equal(got[keep], clean[keep])
    assert S.input_proj_fp8(xq[:0], xs[:0], wq, ws, b).shape == (0, 200)


def test_other_stream(S):
    """Outputs, workspaces and launches belong to the stream that is named."""
    s = torch.cuda.Stream()
    x, w = rand(40, 512, 768, dtype="bf16"), rand(41, 768)
    W = rand(42, 512, 768, scale=0.04)
    torch.cuda.synchronize()
    want = S.rms_norm(x, w, quantize=True)
    Wq, Ws = S.quantize_weight(W)
    y = S.input_proj_fp8(want["y"], want["scale"], Wq, Ws)
    for handle in (s, s.cuda_stream):
        out = S.rms_norm(x, w, quantize=True, stream=handle)
        q = S.quantize_weight(W, stream=handle)
        got = S.input_proj_fp8(out["y"], out["scale"], *q, stream=handle)
        s.synchronize()
        assert torch.equal(got, y)


def test_python_refusals_on_the_device(S):
    x, w = rand(50, 4, 64), rand(51, 64)
    with pytest.raises(ValueError):
        S.rms_norm(x, w[:32])
    with pytest.raises(TypeError):
        S.rms_norm(x.half(), w)
    with pytest.raises(TypeError):
        S.rms_norm(x, w.bfloat16())
    with pytest.raises(ValueError):
        S.rms_norm(x, w, x[:2])
    with pytest.raises(ValueError):
        S.rms_norm(x.T, rand(1, 4))
    with pytest.raises(ValueError):
        S.rms_norm(x, w.cpu())
    with pytest.raises(S.RnnError):
        S.rms_norm(x, w, eps=-1.0)
    xq = torch.zeros(4, 24, device="cuda").to(torch.float8_e4m3fn)
    one = torch.ones(4, 1, device="cuda")
    with pytest.raises(S.RnnError) as e:          # K is no multiple of 16
        S.input_proj_fp8(xq, one, xq, one[:1])
    assert e.value.status == 2
    with pytest.raises(ValueError):
        S.input_proj_fp8(xq, one[:2], xq, one[:1])
