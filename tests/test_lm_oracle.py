"""The fp64 oracle of the language-model operators, pinned on the CPU: closed forms,
and its gradients against central differences."""
import numpy as np
import pytest
import torch

from oracle import lm_oracle as O


def draw(seed, T, B, NH, Dk, Dv):
    r = np.random.default_rng(seed)
    f = lambda *s: r.normal(size=s)  # noqa: E731
    return (f(T, B, NH, Dk), f(T, B, NH, Dk), f(T, B, NH, Dv), -r.uniform(0.01, 1, NH),
            f(T, B, NH, Dv), f(B, NH, Dk, Dv), f(B, NH, Dk, Dv))


def test_linear_attention_is_masked_attention_without_softmax():
    q, k, v, g, _, s0, _ = draw(0, 9, 2, 3, 4, 5)
    o, s = O.linear_attention(q, k, v, g, s0, scale=0.5)
    i = np.arange(9)
    d = np.where(i[:, None] >= i, np.exp(g[:, None, None] * (i[:, None] - i)), 0)  # NH T T
    want = 0.5 * (np.einsum("ibhd,jbhd,hij,jbhe->ibhe", q, k, d, v)
                  + np.einsum("ibhd,bhde,hi->ibhe", q, s0, np.exp(g[:, None] * (i + 1))))
    np.testing.assert_allclose(o, want, rtol=1e-12, atol=1e-12)
    want = np.einsum("jbhd,jbhe,hj->bhde", k, v, np.exp(g[:, None] * (8 - i))) + np.exp(9 * g)[None, :, None, None] * s0
    np.testing.assert_allclose(s, want, rtol=1e-12, atol=1e-12)


def test_linear_attention_rows_without_tokens_and_no_memory():
    q, k, v, g, _, s0, _ = draw(1, 5, 3, 2, 3, 3)
    o, s = O.linear_attention(q, k, v, g, s0, lens=[0, 5, 2])
    assert not o[:, 0].any() and not o[2:, 2].any()
    np.testing.assert_array_equal(s[0], s0[0])
    o, s = O.linear_attention(q, k, v, np.full(2, -np.inf), s0)
    np.testing.assert_allclose(o, np.einsum("tbhd,tbhd->tbh", q, k)[..., None] * v)
    np.testing.assert_allclose(s, np.einsum("bhd,bhe->bhde", k[-1], v[-1]))


@pytest.mark.parametrize("lens", [None, [7, 0, 3]])
def test_linear_attention_gradients_against_differences(lens):
    q, k, v, g, do, s0, ds = draw(2, 7, 3, 2, 3, 4)

    def loss(q, k, v, s0):
        o, s = O.linear_attention(q, k, v, g, s0, lens, 0.7)
        return (o * do).sum() + (s * ds).sum()

    got = O.linear_attention_backward(q, k, v, g, do, s0, ds, lens, 0.7)
    args = [q, k, v, s0]
    r = np.random.default_rng(3)
    for n in range(4):
        d = r.normal(size=args[n].shape)
        hi, lo = (loss(*[a + s * d if i == n else a for i, a in enumerate(args)]) for s in (1, -1))
        # the loss is linear in each argument: the difference over any step is exact
        np.testing.assert_allclose((got[n] * d).sum(), (hi - lo) / 2, rtol=1e-9, atol=1e-9)


def test_rms_norm_gradients_against_differences():
    r = np.random.default_rng(4)
    h, w, dy, dh = r.normal(size=(5, 11)), r.normal(size=11), r.normal(size=(5, 11)), r.normal(size=(5, 11))
    _, rstd = O.rms_norm(h, w, 1e-3)
    dx, dw = O.rms_norm_backward(dy, h, w, rstd, dh)
    f = lambda h, w: (O.rms_norm(h, w, 1e-3)[0] * dy).sum() + (h * dh).sum()  # noqa: E731
    e = 1e-6
    for got, at in ((dx, 0), (dw, 1)):
        d = r.normal(size=got.shape)
        hi, lo = (f(h + s * d, w) if at == 0 else f(h, w + s * d) for s in (e, -e))
        np.testing.assert_allclose((got * d).sum(), (hi - lo) / (2 * e), rtol=1e-7, atol=1e-7)


def test_e4m3_rounding_is_torch_s():
    x = np.concatenate([np.random.default_rng(5).normal(size=4000) * 2.0 ** np.linspace(-12, 9, 4000),
                        np.arange(-464, 465) / 1.0, [0.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 0.0625, 448]])
    x = x.astype(np.float32)
    x = x[np.abs(x) <= 464]  # torch's conversion does not saturate
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(O.e4m3(x), want)


def test_quantize_and_projection():
    r = np.random.default_rng(6)
    y = r.normal(size=(130, 200))
    y[:, :128][3] = 0
    q, s = O.quantize(y)
    assert s.shape == (130, 2) and s[3, 0] == 1 and not q[3, :128].any()
    full = np.repeat(s, 128, 1)[:, :200]
    assert (np.abs(q * full - y) <= 2.0 ** -4 * np.abs(y) + full * 2.0 ** -10 + 1e-15).all()
    wq, ws = O.quantize(y, 128)
    assert ws.shape == (2, 2)
    got, mag = O.proj_fp8(q[:4], s[:4], wq, ws, np.ones(130))
    w = wq * np.repeat(np.repeat(ws, 128, 0)[:130], 128, 1)[:, :200]
    np.testing.assert_allclose(got, (q[:4] * full[:4]) @ w.T + 1, rtol=1e-12)
    assert (mag >= np.abs(got) - 1e-9).all()
