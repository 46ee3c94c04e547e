"""The fp64 oracle of the gated recurrence, the head norm with rotation and the clipping, against automatic
differentiation of their definitions, closed forms and invariants."""
import numpy as np
import pytest
import torch

from oracle import mix_oracle as O


def rnd(seed, *shape):
    return np.random.default_rng(seed).normal(size=shape)


def torch_gated(Wx, gates, s0, lens):
    T, B = Wx.shape[:2]
    p = dict(zip(gates, Wx.unflatten(-1, (len(gates), -1)).unbind(-2)))
    f = torch.sigmoid(p["f"])
    gain = torch.sigmoid(p["i"]) if "i" in p else 1 - f
    c, ys = s0, []
    for t in range(T):
        on = (torch.tensor(lens) > t)[:, None, None]
        c = torch.where(on, f[t] * c + gain[t] * p["z"][t], c)
        ys.append(torch.where(on, c * torch.sigmoid(p["o"][t]) if "o" in p else c, torch.zeros(())))
    return torch.stack(ys), c


@pytest.mark.parametrize("gates", ["fz", "fzo", "ifzo"])
def test_gated_against_autograd(gates):
    T, B, NH, D, lens = 13, 4, 2, 3, [13, 0, 7, 20]
    Wx = torch.from_numpy(rnd(1, T, B, NH, len(gates) * D)).requires_grad_()
    s0 = torch.from_numpy(rnd(2, B, NH, D)).requires_grad_()
    dy, ds = rnd(3, T, B, NH, D), rnd(4, B, NH, D)
    y, c = torch_gated(Wx, gates, s0, lens)
    ((y * torch.from_numpy(dy)).sum() + (c * torch.from_numpy(ds)).sum()).backward()
    f = O.gated(Wx.detach().numpy(), gates, s0.detach().numpy(), lens)
    g = O.gated_backward(Wx.detach().numpy(), gates, dy, s0.detach().numpy(), ds, lens)
    for got, want in ((f["y"], y), (f["state"], c), (g["dWx"], Wx.grad), (g["dstate"], s0.grad)):
        np.testing.assert_allclose(got, want.detach().numpy(), rtol=1e-12, atol=1e-13)


@pytest.mark.parametrize("gates", ["fz", "ifzo"])
def test_gated_gradient_against_differences(gates):
    T, B, NH, D = 6, 1, 1, 2
    Wx, s0, dy, ds = rnd(1, T, B, NH, len(gates) * D), rnd(2, B, NH, D), rnd(3, T, B, NH, D), rnd(4, B, NH, D)

    def loss(w, s):
        f = O.gated(w, gates, s)
        return (f["y"] * dy).sum() + (f["state"] * ds).sum()

    g, h = O.gated_backward(Wx, gates, dy, s0, ds), 1e-5
    for x, grad, at in ((Wx, g["dWx"], lambda v: loss(v, s0)), (s0, g["dstate"], lambda v: loss(Wx, v))):
        for i in np.ndindex(*x.shape):
            up, dn = x.copy(), x.copy()
            up[i] += h
            dn[i] -= h
            assert abs((at(up) - at(dn)) / (2 * h) - grad[i]) <= 1e-8


def test_gated_bounds_hold_for_fp32():
    """The same recurrence in numpy fp32 stays within the bounds."""
    T, B, NH, D = 400, 2, 1, 16
    Wx = rnd(5, T, B, NH, 2 * D).astype(np.float32)
    Wx[..., :D] += 4
    f = O.gated(Wx, "fz")
    e = np.exp(-np.abs(Wx[..., :D]))
    low = e / (np.float32(1) + e)
    a = np.where(Wx[..., :D] > 0, np.float32(1) - low, low)
    u = np.where(Wx[..., :D] > 0, low, np.float32(1) - low) * Wx[..., D:]
    c = np.zeros((B, NH, D), np.float32)
    for t in range(T):
        c = a[t] * c + u[t]
        assert (np.abs(c - f["c"][t + 1]) <= f["c_err"][t + 1]).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 4, 8])
def test_rotary_against_autograd(rot, interleaved):
    T, B, H, D = 5, 2, 3, 8
    x = torch.from_numpy(rnd(1, T, B, H, D)).requires_grad_()
    w = torch.from_numpy(1 + 0.1 * rnd(2, D)).requires_grad_()
    freqs, at, dy = np.abs(rnd(3, rot // 2)), np.array([3, 100]), rnd(4, T, B, H, D)
    y = x / (x.pow(2).mean(-1, keepdim=True) + 1e-5).sqrt() * w
    ang = torch.from_numpy((at[None] + np.arange(T)[:, None])[..., None] * freqs)[:, :, None]
    a, b = (list(range(0, rot, 2)), list(range(1, rot, 2))) if interleaved else (list(range(rot // 2)), list(range(rot // 2, rot)))
    rows = [None] * D
    for j, (ia, ib) in enumerate(zip(a, b)):
        c, s = torch.cos(ang[..., j]), torch.sin(ang[..., j])
        rows[ia], rows[ib] = y[..., ia] * c - y[..., ib] * s, y[..., ib] * c + y[..., ia] * s
    out = torch.stack([y[..., i] if r is None else r for i, r in enumerate(rows)], -1)
    (out * torch.from_numpy(dy)).sum().backward()
    got, _ = O.head_norm_rotary(x.detach().numpy(), w.detach().numpy(), freqs, at, 1e-5, interleaved)
    np.testing.assert_allclose(got, out.detach().numpy(), rtol=1e-12, atol=1e-13)
    dx, _, dw, _ = O.head_norm_rotary_backward(x.detach().numpy(), w.detach().numpy(), freqs, at, dy, 1e-5, interleaved)
    np.testing.assert_allclose(dx, x.grad.numpy(), rtol=1e-11, atol=1e-12)
    np.testing.assert_allclose(dw, w.grad.numpy(), rtol=1e-11, atol=1e-12)


def test_rotary_products_depend_on_the_distance():
    q, k = rnd(1, 1, 1, 1, 16), rnd(2, 1, 1, 1, 16)
    freqs = 10000.0 ** (-np.arange(8) / 8)
    dots = [(O.head_norm_rotary(q, None, freqs, np.array([s + 7]), 0, False)[0]
             * O.head_norm_rotary(k, None, freqs, np.array([s]), 0, False)[0]).sum() for s in (0, 5, 100000, -3)]
    np.testing.assert_allclose(dots, dots[0], rtol=1e-10)


def test_clip():
    x = [np.array([3.0]), np.array([[0.0, 4.0]])]
    norm, out = O.clip(x, 1.0)
    assert norm == 5.0 and out[1][0, 1] == pytest.approx(0.8)
    assert O.clip(x, 5.0)[1][0][0] == 3.0 and O.clip([np.array([np.inf, 1.0])], 1.0)[1][0][1] == 1.0
