"""GPU tests of the 8-bit norm where its values are not ordinary numbers, against the definition in 64 bits.

The codes are those of 448 h w / max|h w|, rounded to fp32 and then to e4m3: compared exactly.
"""
import numpy as np
import pytest
import torch

from oracle import lm_oracle as O

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# a row in a warp's vectors, in a CTA's, value by value in registers, and past what they hold
WIDTHS = [256, 1000, 8192, 301, 5001]


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


def blocks(a):
    """[rows, N] -> [rows, blocks, 128], zeros behind the row's end."""
    return np.pad(a, ((0, 0), (0, -a.shape[1] % 128))).reshape(a.shape[0], -1, 128)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", WIDTHS)
@pytest.mark.parametrize("where", ["column", "among zeros", "block", "all"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_weights_that_are_not_finite(S, N, where, value, dtype):
    """A product that is not a number has a NaN code and does not count towards its block's scale; an infinite one has
    a NaN code and an infinite scale.  The other blocks do not notice."""
    rows = 5
    x, w = rand(1, rows, N, dtype=dtype), rand(2, N)
    lo = 128
    hit = {"column": slice(lo + 3, lo + 4), "among zeros": slice(lo + 3, lo + 4), "block": slice(lo, lo + 128),
           "all": slice(0, N)}[where]
    if where == "among zeros":
        x[:, lo:lo + 128] = 0
        x[:, lo + 3] = 1
    w[hit] = value
    out = S.rms_norm(x, w, quantize=True)
    y, scale = np64(out["y"]), np64(out["scale"])
    with np.errstate(invalid="ignore"):
        hw = np64(x) * np64(w)
    mag = blocks(np.where(np.isnan(hw), 0, np.abs(hw)))
    top = mag.max(2)
    assert np.array_equal(np.isnan(y), ~np.isfinite(hw))
    assert np.array_equal(np.isinf(scale), np.isinf(top)) and (scale[top == 0] == 1).all()
    ok = np.isfinite(top) & (top > 0)
    full = np.repeat(np.where(ok, top, 1), 128, 1)[:, :N]
    fine = np.isfinite(hw) & np.repeat(np.isfinite(top), 128, 1)[:, :N]
    want = O.e4m3((448 * np.where(fine, hw, 0) / full).astype(np.float32))
    assert np.array_equal(y[fine], want[fine])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [256, 1000, 301])
def test_a_subnormal_scale_between_factors_that_are_not(S, N, dtype):
    """A column of some 2^64 makes rstd 2^-59, a block's largest product is 2^-59, and its scale, 2^-127, is subnormal: coarse.
    The codes are of the quotient by what is stored.  The products are ties of the quotient by the scale
    before it was rounded, which fall to either side as the rounding goes."""
    rows = 40
    x = torch.zeros(rows, N)
    x[:, 0] = 2.0 ** 63 * (1.5 + torch.arange(rows) / 128)
    x[:, 128:256] = torch.tensor([448, 272, -304, 336, 368, -400, 432, 136] * 16)
    w = torch.ones(N)
    w[128:256] = 2.0 ** -68
    x, w = x.to(DT[dtype]).cuda(), w.cuda()
    out = S.rms_norm(x, w, quantize=True, train=True)
    s = np64(out["scale"])[:, 1:2]
    assert (s < 2.0 ** -126).all() and (s > 2.0 ** -129).all() and (np64(out["rstd"]) > 2.0 ** -60).all()
    q = np64(x)[:, 128:256] * np64(w)[128:256] * (np64(out["rstd"])[:, None] / s)
    assert np.array_equal(np64(out["y"])[:, 128:256], O.e4m3(q.astype(np.float32)))


def codes(h, w):
    """e4m3 of the quotient by the block's scale, as rnn_rms_norm defines it."""
    hw = np64(h) * np64(w)
    top = blocks(np.abs(hw)).max(2)
    top = np.repeat(np.where(top > 0, top, 1), 128, 1)[:, :hw.shape[1]]
    return O.e4m3((448 * hw / top).astype(np.float32))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("weights", ["drawn", "ones"])
@pytest.mark.parametrize("rows,N", [(1, 1), (5, 1), (3, 2), (3, 7), (2, 8), (300, 8), (40, 9), (33, 100), (20, 120), (21, 127),
                                    (19, 128), (17, 129), (16, 136), (9, 255), (9, 257)])
def test_codes_of_narrow_rows(S, rows, N, weights, dtype):
    """A block that ends early, blocks of a few columns, rows narrower than a vector: equal codes."""
    x, res, w = rand(70, rows, N, dtype=dtype), rand(71, rows, N, dtype=dtype), rand(72, N)
    if weights == "ones":                          # products of 8 bits: many exact ties
        w = torch.ones_like(w)
    out = S.rms_norm(x, w, res, quantize=True)
    assert np.array_equal(np64(out["y"]), codes(out["h"], w))
    y, _ = O.rms_norm(np64(out["h"]), np64(w), 1e-6)
    np.testing.assert_allclose(np64(out["scale"]), O.quantize(y)[1], rtol=2.0 ** -20)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,K", [(1, 1), (1, 7), (7, 1), (2, 129), (129, 2), (128, 128), (130, 300), (5, 1000)])
def test_weight_codes(S, N, K, dtype):
    """A code is that of W over the stored scale, unless the quotient lies within fp32's error (2^-23 of it) of a tie."""
    W = rand(73, N, K, dtype=dtype)
    W[:, ::5] = W[:, ::5].bfloat16().to(W.dtype)
    Wq, Ws = S.quantize_weight(W)
    s = np.repeat(np.repeat(np64(Ws), 128, 0)[:N], 128, 1)[:, :K]
    top = O.quantize(np64(W), 128)[1]
    np.testing.assert_allclose(np64(Ws), top, rtol=2.0 ** -23)
    q = np64(W) / s
    lo, hi = O.e4m3(q * (1 - 2.0 ** -23)), O.e4m3(q * (1 + 2.0 ** -23))
    got = np64(Wq)
    assert ((got == lo) | (got == hi)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_weights_to_quantise_that_are_not_finite(S, dtype):
    """As in the norm: NaN codes; a NaN leaves its block's scale to the others, an infinity makes it infinite."""
    W = rand(74, 300, 400, dtype=dtype)
    clean = S.quantize_weight(W)
    W[5, 7], W[140, 390], W[130, 150] = float("nan"), float("inf"), -float("inf")
    W[256:300, 256:384] = float("nan")             # a whole block
    q, s = S.quantize_weight(W)
    bad = ~torch.isfinite(W)
    assert torch.equal(q.float().isnan(), bad)
    want = clean[1].clone()
    want[0, 0] = W[:128, :128][~bad[:128, :128]].float().abs().max() / 448
    want[1, 3], want[1, 1], want[2, 2] = float("inf"), float("inf"), 1.0
    assert torch.allclose(s, want, rtol=2.0 ** -22, atol=0)
    other = torch.ones_like(bad)
    for i, j in ((0, 0), (1, 3), (1, 1), (2, 2)):
        other[128 * i:128 * i + 128, 128 * j:128 * j + 128] = False
    assert torch.equal(q.float()[other], clean[0].float()[other])
