"""GPU tests of the gated recurrence, the head norm with rotation and the clipping on tensors of more than 2^31 values: what
stands behind their 32-bit counts is compared with the fp64 oracle.  Tolerances as in the operators' own tests."""
import numpy as np
import pytest
import torch

from oracle import mix_oracle as O

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -8


@pytest.fixture(scope="module")
def S():
    from sequential_rnn_gb300 import build
    build.build()
    import sequential_rnn_gb300 as S
    if torch.cuda.get_device_properties(0).total_memory < 60 << 30:
        pytest.skip("needs 60 GB")
    yield S
    torch.cuda.empty_cache()


def np64(t):
    return t.detach().double().cpu().numpy()


def randn(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


@pytest.mark.parametrize("D", [256, 257])  # on tiles, and value by value
def test_gated(S, D):
    T, B, NH = 3000, 200, 7
    Wx = randn(1, T, B, NH, 2 * D)
    assert Wx.numel() > 2 ** 31
    dy = randn(2, T, B, NH, D)
    out = S.gated_recurrence(Wx, train=True)
    g = S.gated_recurrence_backward(Wx, out["stash"], dy)
    cols = [0, D - 1]
    wx = np64(Wx[:, -1:, -1:].reshape(T, 1, 1, 2, D)[..., cols].reshape(T, 1, 1, 4))
    f = O.gated(wx, "fz", fast=True)
    b = O.gated_backward(wx, "fz", np64(dy[:, -1:, -1:, cols]), fast=True)
    y, dw = np64(out["y"][:, -1:, -1:, cols]), np64(g["dWx"][:, -1:, -1:].reshape(T, 1, 1, 2, D)[..., cols]).reshape(T, 1, 1, 4)
    assert (np.abs(y - f["y"]) <= f["y_err"] + HALF * 1.001 * np.abs(f["y"]) + 1e-30).all()
    assert (np.abs(np64(out["state"][-1:, -1:, cols]) - f["state"]) <= f["state_err"] + 1e-7 * np.abs(f["state"])).all()
    assert (np.abs(dw - b["dWx"]) <= b["dWx_err"] * 1.01 + HALF * 1.001 * np.abs(b["dWx"]) + 1e-30).all()


def test_rotary(S):
    T, B, NH, D = 4100, 64, 64, 128
    q = randn(1, T, B, NH, D)
    assert q.numel() > 2 ** 31
    k, w, f = q[:, :, :2], 1 + 0.1 * randn(2, D).float(), S.rotary_frequencies(D)
    at = torch.arange(B, dtype=torch.int32, device="cuda")
    yq, yk = S.head_norm_rotary(q, k, w, w, f, at)
    g = S.head_norm_rotary_backward(q, k, w, w, f, at, q, k)
    last = np64(q[-1:, -1:])
    y, err = O.head_norm_rotary(last, np64(w), np64(f), np.array([[B - 1 + T - 1]]), 1e-6, False)
    assert (np.abs(np64(yq[-1:, -1:]) - y) <= err + HALF * 1.001 * np.abs(y) + 1e-30).all()
    assert torch.equal(yk[-1], yq[-1, :, :2])
    dx, dxe, _, _ = O.head_norm_rotary_backward(last, np64(w), np64(f), np.array([[B - 1 + T - 1]]), last, 1e-6, False)
    assert (np.abs(np64(g["dq"][-1:, -1:]) - dx) <= dxe + HALF * 1.001 * np.abs(dx) + 1e-30).all()
    assert torch.equal(g["dk"][-1], g["dq"][-1, :, :2])


def test_clip(S):
    n = 2 ** 31 + 4099
    x = randn(1, n)
    keep = x[-5000:].clone()
    norm = np.sqrt(sum(float(c.double().square().sum()) for c in x.split(1 << 27)))
    got = S.clip_grad_norm([x], 1.0).item()
    assert abs(got - norm) <= 17 * 2.0 ** -24 * norm
    want = np64(keep) / norm
    assert (np.abs(np64(x[-5000:]) - want) <= (HALF + 24 * 2.0 ** -24) * np.abs(want)).all()
    assert S.grad_norm([x]).item() == pytest.approx(1.0, rel=2.0 ** -8)
