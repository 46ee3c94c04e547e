"""The gated recurrence, the head norm with rotation and the clipping as examples/linear_attention_lm.py runs them, beside the
norm, the 8-bit projection and linear attention: the stack's outputs against the fp64 oracle of the same layers, single
tokens against the prompt, and a training step's gradients against automatic differentiation in fp64.

Tolerances, as a ratio of norms: each 8-bit rounding point leaves sqrt(2^-8 2^-3) = 0.022 (a value that differs by a
fraction d before an e4m3 rounding falls to the other side with a probability of d / 2^-3 and then differs by
2^-3; bf16 results carry 2^-8 at most).  A stack of a rotary and a gated layer has three of them in a row, 0.066
if all add up.  The training step has no 8-bit rounding: bf16 roundings of the norm's output, the turned
queries and keys, scores, states, the attention's gradients, the rotation's, the gates' and dx: ten of 2^-8 at most.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import lm_oracle as O
from oracle import mix_oracle as MO

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TOL8, TOL16 = 0.066, 10 * 2.0 ** -8


@pytest.fixture(scope="module")
def ex():
    from sequential_rnn_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("linear_attention_lm",
                                                  os.path.join(ROOT, "examples", "linear_attention_lm.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def np64(t):
    return t.detach().double().cpu().numpy()


def ratio(got, want):
    return np.linalg.norm(got - want) / np.linalg.norm(want)


def oracle_prompt(m, x, lens):
    """The model's prompt in fp64, 8-bit roundings included."""
    T, B, d = x.shape
    flat = lambda t: t.reshape(T * B, -1)  # noqa: E731

    def proj(y, w, bias=0.0):
        return (O.proj_fp8(*O.quantize(flat(y)), *O.quantize(np64(w), 128))[0] + bias).reshape(T, B, -1)

    norm = lambda h, w: O.rms_norm(flat(h), np64(w), 1e-6)[0].reshape(h.shape)  # noqa: E731
    out = np.zeros_like(x)
    for layer in m.layers:
        x = x + out
        if hasattr(layer, "bias"):
            wx = proj(norm(x, layer.n), layer.w, np64(layer.bias).reshape(-1)).reshape(T, B, layer.NH, -1)
            out = MO.gated(wx, "fzo", lens=lens)["y"].reshape(T, B, d)
        else:
            q, k, v = proj(norm(x, layer.n_in), layer.w_in).reshape(T, B, 3, layer.NH, layer.D).transpose(2, 0, 1, 3, 4)
            q, k = (MO.head_norm_rotary(t, np64(w), np64(layer.freqs), None, 1e-6, False)[0]
                    for t, w in ((q, layer.n_q), (k, layer.n_k)))
            o, _ = O.linear_attention(q, k, v, np64(layer.decay), lens=lens, scale=layer.D ** -0.5)
            out = proj(norm(o.reshape(T, B, d), layer.n_out), layer.w_out)
    return norm(x + out, m.norm)


@pytest.mark.parametrize("lens", [None, [150, 64, 1]])
def test_prompt_against_oracle(ex, lens):
    NH, D, B, T = 2, 64, 3, 150
    m = ex.Model(NH, D, layers=("rotary", "gated"), seed=3)
    x = torch.randn(T, B, NH * D, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    y, _ = m.prompt(x, None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda"))
    want = oracle_prompt(m, np64(x), lens)
    for b, n in enumerate(lens or [T] * B):
        assert ratio(np64(y)[:n, b], want[:n, b]) <= TOL8


@pytest.mark.parametrize("graph", [False, True])
def test_steps_continue_the_prompt(ex, graph):
    NH, D, B, T, T0 = 2, 64, 3, 90, 71
    m = ex.Model(NH, D, layers=("rotary", "gated"), seed=5)
    x = torch.randn(T, B, NH * D, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    want, _ = m.prompt(x)
    y, caches = m.prompt(x[:T0])
    got = []
    if graph:
        xin, yout, replay = m.graph(caches, B)
    for t in range(T0, T):
        if graph:
            xin.copy_(x[t])
            replay()
            got.append(yout.clone())
        else:
            got.append(m.step(x[t], caches))
    assert ratio(np64(torch.stack(got)), np64(want[T0:])) <= TOL8


@pytest.mark.parametrize("limit", [1e-3, 1e9])
def test_training_step_against_autograd(ex, limit):
    NH, D, B, T = 2, 64, 2, 100
    d = NH * D
    g = torch.Generator().manual_seed(3)
    x = torch.randn(T, B, 5 * d, generator=g).bfloat16()
    w, wq, wk = (1 + 0.1 * torch.randn(n, generator=g) for n in (5 * d, D, D))
    target = torch.randn(T, B, NH, D, generator=g).bfloat16()
    freqs, decay = ex.S.rotary_frequencies(D), ex.decays(NH)
    _, grads, dx, norm = ex.training_step(x.cuda(), w.cuda(), wq.cuda(), wk.cuda(), freqs, decay, NH, D, target.cuda(), limit)

    X, W, WQ, WK = (t.double().requires_grad_() for t in (x, w, wq, wk))
    y = X * torch.rsqrt((X * X).mean(-1, keepdim=True) + 1e-6) * W
    q, k, v = y[..., :3 * d].reshape(T, B, 3, NH, D).unbind(2)
    ang = (torch.arange(T, dtype=torch.float64)[:, None] * freqs.cpu())[:, None, None]

    def turned(t, weight):
        t = t * torch.rsqrt((t * t).mean(-1, keepdim=True) + 1e-6) * weight
        a, b = t[..., :D // 2], t[..., D // 2:]
        return torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)

    lag = torch.arange(T)[:, None] - torch.arange(T)[None]
    mask = torch.where(lag >= 0, torch.exp(decay.double().cpu()[:, None, None] * lag.clamp(min=0)), 0.0)
    o = torch.einsum("hts,bhts,sbhe->tbhe", mask, torch.einsum("tbhd,sbhd->bhts", turned(q, WQ), turned(k, WK)), v) * D ** -0.5
    f, z = y[..., 3 * d:].reshape(T, B, NH, 2, D).unbind(3)
    f, c, ys = torch.sigmoid(f), torch.zeros(B, NH, D, dtype=torch.float64), []
    for t in range(T):
        c = f[t] * c + (1 - f[t]) * z[t]
        ys.append(c)
    ((o + torch.stack(ys)) * target.double()).sum().backward()
    assert ratio(np64(dx), X.grad.numpy()) <= TOL16
    want = [W.grad.numpy(), WQ.grad.numpy(), WK.grad.numpy()]
    n64, clipped = MO.clip(want, limit)
    assert abs(norm.item() - n64) <= TOL16 * n64
    got = np.concatenate([np64(t) for t in grads.values()])
    assert ratio(got, np.concatenate(clipped)) <= 2 * TOL16  # (the gradients' error and the factor's)
    assert ex.S.grad_norm(list(grads.values())).item() <= max(limit, 0) * (1 + 2.0 ** -20) or limit > n64
