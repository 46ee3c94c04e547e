"""The operators together, as examples/linear_attention_lm.py runs them: the stack's outputs against the fp64
oracle of the same layers, single tokens against the prompt, and the gradient of norm and linear attention
against automatic differentiation in fp64.

Tolerances, as a ratio of norms.  A value that differs by a fraction d before an e4m3 rounding
(spacing up to 2^-3 of the value) falls to the other side with a probability of about d / 2^-3 and then
differs by 2^-3: root mean square sqrt(d 2^-3).  bf16 results carry d ~ 2^-9 (root mean square 2^-9
of an element or less, two of them 2^-8), so that each 8-bit rounding point leaves sqrt(2^-8 2^-3) = 0.022;
the stack of three layers has five such points, in a row along the residual stream: at most
0.11 if all of them add up, 0.05 if they are independent.  The bound is 0.11.  The gradient has no 8-bit
rounding: bf16 roundings of y, q k v's scores, states, gradients and the result, eight of 2^-8 at most.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import lm_oracle as O
from oracle import rnn_oracle as RO

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TOL8, TOL16 = 0.11, 8 * 2.0 ** -8


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
    return t.detach().float().cpu().numpy().astype(np.float64)


def ratio(got, want):
    return np.linalg.norm(got - want) / np.linalg.norm(want)


def oracle_prompt(m, x):
    """The model's prompt in fp64, 8-bit roundings included."""
    T, B, d = x.shape
    flat = lambda t: t.reshape(T * B, -1)  # noqa: E731

    def proj(y, w):
        return O.proj_fp8(*O.quantize(flat(y)), *O.quantize(np64(w), 128))[0].reshape(T, B, -1)

    norm = lambda h, w: O.rms_norm(flat(h), np64(w), 1e-6)[0].reshape(h.shape)  # noqa: E731
    out = np.zeros_like(x)
    for layer in m.layers:
        x = x + out
        if hasattr(layer, "R"):
            wx = proj(norm(x, layer.n), layer.w).reshape(T, B, layer.NH, -1)
            out = RO.forward("lstm", wx, np64(layer.R))["h_seq"].reshape(T, B, d)
        else:
            qkv = proj(norm(x, layer.n_in), layer.w_in).reshape(T, B, 3, layer.NH, layer.D)
            o, _ = O.linear_attention(*qkv.transpose(2, 0, 1, 3, 4), np64(layer.decay),
                                      scale=layer.D ** -0.5)
            out = proj(norm(o.reshape(T, B, d), layer.n_out), layer.w_out)
    return norm(x + out, m.norm)


@pytest.mark.parametrize("NH,D,B,T", [(2, 64, 3, 150), (3, 32, 2, 70)])
def test_prompt_against_oracle(ex, NH, D, B, T):
    m = ex.Model(NH, D, seed=NH)
    x = torch.randn(T, B, NH * D, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    y, _ = m.prompt(x)
    assert ratio(np64(y), oracle_prompt(m, np64(x))) <= TOL8


@pytest.mark.parametrize("graph", [False, True])
def test_steps_continue_the_prompt(ex, graph):
    NH, D, B, T, T0 = 2, 64, 3, 90, 71
    m = ex.Model(NH, D, seed=5)
    x = torch.randn(T, B, NH * D, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    want, _ = m.prompt(x)
    y, caches = m.prompt(x[:T0])
    assert ratio(np64(y), np64(want[:T0])) <= TOL8
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


def test_gradient_against_autograd(ex):
    NH, D, B, T = 2, 64, 2, 100
    g = torch.Generator().manual_seed(3)
    x = torch.randn(T, B, 3 * NH * D, generator=g).bfloat16()
    w = 1 + 0.1 * torch.randn(3 * NH * D, generator=g)
    target = torch.randn(T, B, NH, D, generator=g).bfloat16()
    decay = ex.decays(NH)
    _, dx, dw = ex.mixer_loss(x.cuda(), w.cuda(), decay, NH, D, target.cuda())

    X, Wt = x.double().requires_grad_(), w.double().requires_grad_()
    y = X * torch.rsqrt((X * X).mean(-1, keepdim=True) + 1e-6) * Wt
    q, k, v = y.view(T, B, 3, NH, D).unbind(2)
    lag = torch.arange(T)[:, None] - torch.arange(T)[None]
    decay = decay.double().cpu()
    mask = torch.where(lag >= 0, torch.exp(decay[:, None, None] * lag.clamp(min=0)), 0.0)
    o = torch.einsum("hts,bhts,sbhe->tbhe", mask, torch.einsum("tbhd,sbhd->bhts", q, k), v) * D ** -0.5
    (o * target.double()).sum().backward()
    assert ratio(np64(dx), X.grad.numpy()) <= TOL16
    assert ratio(np64(dw), Wt.grad.numpy()) <= TOL16
