"""fp64 oracle of the gated linear recurrence (token by token), the norm and rotation of heads and the
clipping of gradients, with bounds of what fp32 arithmetic may change.  Test infrastructure (numpy)."""
from __future__ import annotations

import math

import numpy as np

__all__ = ["gated", "gated_backward", "head_norm_rotary", "head_norm_rotary_backward", "clip"]
E = 2.0 ** -24  # half a step of fp32, relative


def _sigmoids(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x)), 1.0 / (1.0 + np.exp(x))


def _lens(T, B, lens):
    return np.full(B, T) if lens is None else np.clip(np.asarray(lens), 0, T)


def _split(Wx, gates):
    x = np.asarray(Wx, np.float64)
    x = x.reshape(*x.shape[:-1], len(gates), x.shape[-1] // len(gates))
    return {n: x[..., i, :] for i, n in enumerate(gates)}


def gated(Wx, gates, state=None, lens=None, fast=False):
    """Wx [T,B,NH,G*D] -> dict of y, state (the last), c [T+1,B,NH,D] (all states) and the bounds y_err, state_err,
    c_err of fp32 arithmetic.

    A step c = a c + u: a's error is at most 8 E of sigm(-f) (exponential, quotient) and E of itself, u's 10 E; the step's
    sum is rounded once and the products of a that carry a state over several tokens once and a half a token.
    fast (bf16 gates): e^-|x| as 2^t with t = |x| log2 e rounded to fp32, off by at most 2 |x| E more (the product's
    rounding, 2^-24 of t, and the constant's, 2^-25, both times log 2)."""
    p = _split(Wx, gates)
    more = {n: 2 * np.abs(p[n]) if fast and n != "z" else 0.0 * p[n] for n in p}
    T, B, NH, D = p["f"].shape
    (a, low), z = _sigmoids(p["f"]), p["z"]
    gain = _sigmoids(p["i"])[0] if "i" in p else low
    o = _sigmoids(p["o"])[0] if "o" in p else np.ones_like(a)
    live = (np.arange(T)[:, None] < _lens(T, B, lens)[None])[..., None, None]
    c = np.zeros((T + 1, B, NH, D))
    if state is not None:
        c[0] = state
    m, err = np.abs(c[0]), np.zeros((T + 1, B, NH, D))
    for t in range(T):
        u = gain[t] * z[t]
        c[t + 1] = np.where(live[t], a[t] * c[t] + u, c[t])
        k = 10 + more["i" if "i" in p else "f"][t]
        new = a[t] * err[t] + E * (4 + (8 + more["f"][t]) * low[t]) * a[t] * m + k * E * np.abs(u)
        err[t + 1] = np.where(live[t], new, err[t])
        m = np.where(live[t], a[t] * m + np.abs(u), m)
    y = np.where(live, o * c[1:], 0.0)
    return {"y": y, "state": c[T], "c": c, "state_err": err[T], "c_err": err,
            "y_err": np.where(live, o * err[1:] + ((12 + more["o"]) * E if "o" in p else 0.0) * np.abs(y), 0.0)}


def gated_backward(Wx, gates, dy, state=None, dstate=None, lens=None, fast=False):
    """dWx and the initial state's gradient of sum(y dy) + sum(state dstate), with their bounds."""
    p = _split(Wx, gates)
    T, B, NH, D = p["f"].shape
    f = gated(Wx, gates, state, lens, fast)
    more = {n: 2 * np.abs(p[n]) if fast and n != "z" else 0.0 * p[n] for n in p}
    mo, mg = more.get("o", np.zeros_like(p["f"])), more["i" if "i" in p else "f"]
    c, ec = f["c"], f["c_err"]
    (a, low), z = _sigmoids(p["f"]), p["z"]
    gain, gainc = _sigmoids(p["i"]) if "i" in p else (low, a)
    o, oc = _sigmoids(p["o"]) if "o" in p else (np.ones_like(a), np.zeros_like(a))
    live = (np.arange(T)[:, None] < _lens(T, B, lens)[None])[..., None, None]
    dy = np.where(live, np.asarray(dy, np.float64), 0.0)
    d = np.zeros((B, NH, D)) if dstate is None else np.array(dstate, np.float64)  # a_{t+1} dc_{t+1}
    m, err = np.abs(d), np.zeros_like(d)
    g = {n: np.zeros_like(a) for n in gates}
    ge = {n: np.zeros_like(a) for n in gates}
    for t in reversed(range(T)):
        e = dy[t] * o[t]
        dc, edc = d + e, err + (12 + mo[t]) * E * np.abs(e) + E * m
        mc = m + np.abs(e)
        g["z"][t] = dc * gain[t]
        ge["z"][t] = (edc + (12 + mg[t]) * E * np.abs(dc)) * gain[t]
        x = c[t] if "i" in p else c[t] - z[t]
        ex = ec[t] + E * (np.abs(c[t]) + np.abs(z[t]))
        s = a[t] * low[t]
        g["f"][t] = dc * x * s
        ge["f"][t] = s * (edc * np.abs(x) + np.abs(dc) * ex + (24 + 2 * more["f"][t]) * E * np.abs(dc * x))
        if "i" in p:
            g["i"][t] = dc * z[t] * gain[t] * gainc[t]
            ge["i"][t] = gain[t] * gainc[t] * np.abs(z[t]) * (edc + (24 + 2 * more["i"][t]) * E * np.abs(dc))
        if "o" in p:
            # (the state after the token, formed once more from the one before it)
            g["o"][t] = dy[t] * c[t + 1] * o[t] * oc[t]
            ge["o"][t] = o[t] * oc[t] * np.abs(dy[t]) * (ec[t + 1] + (24 + 2 * mo[t]) * E * np.abs(c[t + 1]))
        d = np.where(live[t], a[t] * dc, d)
        err = np.where(live[t], a[t] * edc + E * (4 + (8 + more["f"][t]) * low[t]) * a[t] * mc, err)
        m = np.where(live[t], a[t] * mc, m)
    stack = lambda q: np.where(live, np.stack([q[n] for n in gates], -2).reshape(T, B, NH, len(gates) * D), 0.0)  # noqa: E731
    return {"dWx": stack(g), "dWx_err": stack(ge), "dstate": d, "dstate_err": err}


def _cos_sin(T, B, freqs, positions):
    """[T, B, 1, rot/2]; the angle in extended precision (a far position's fp64 product would be off by as much as
    the kernel may be)."""
    t = np.arange(T)[:, None]
    if positions is None:
        at = t + np.zeros((1, B), np.int64)
    else:
        at = np.asarray(positions).astype(np.int64)
        at = at[None] + t if at.ndim == 1 else at
    x = at.astype(np.longdouble)[..., None] * np.asarray(freqs, np.float64).astype(np.longdouble)
    return np.cos(x).astype(np.float64)[:, :, None], np.sin(x).astype(np.float64)[:, :, None]


def _pairs(D, rot, interleaved):
    j = np.arange(rot // 2)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)


def _turn(x, cos, sin, interleaved):
    a, b = _pairs(x.shape[-1], 2 * cos.shape[-1], interleaved)
    y = x.copy()
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def head_norm_rotary(x, w, freqs, positions, eps, interleaved):
    """x [T,B,H,D] -> (y, bound): the norm's relative error is (D/32 + 12) E, an angle's 8 E (its fraction of a turn is
    rounded to 24 bits, then the sine's and cosine's own error)."""
    x = np.asarray(x, np.float64)
    T, B, _, D = x.shape
    cos, sin = _cos_sin(T, B, np.zeros(0) if freqs is None else freqs, positions)
    y = x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    mag = _turn(np.abs(y), np.ones_like(cos), -np.ones_like(sin), interleaved)  # |y1| + |y2| at y1
    a, b = _pairs(D, 2 * cos.shape[-1], interleaved)
    mag[..., b] = mag[..., a]
    return _turn(y, cos, sin, interleaved), (D / 32 + 20) * E * mag


def head_norm_rotary_backward(x, w, freqs, positions, dy, eps, interleaved):
    """(dx, its bound, dw, its bound); dw None without weights."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    T, B, H, D = x.shape
    cos, sin = _cos_sin(T, B, np.zeros(0) if freqs is None else freqs, positions)
    g = _turn(dy, cos, -sin, interleaved)
    mag = _turn(np.abs(dy), np.ones_like(cos), -np.ones_like(sin), interleaved)
    a, b = _pairs(D, 2 * cos.shape[-1], interleaved)
    mag[..., b] = mag[..., a]
    if w is None:
        return g, 20 * E * mag, None, None
    w = np.asarray(w, np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * r
    dx = r * (w * g - xh * (w * g * xh).mean(-1, keepdims=True))
    k = (D / 16 + 40) * E
    dxe = k * r * (np.abs(w) * mag + np.abs(xh) * (np.abs(w) * mag * np.abs(xh)).mean(-1, keepdims=True))
    n = T * B * H  # a sum of n terms in pieces: at most sqrt-like growth is not relied on
    dw = (g * xh).sum((0, 1, 2))
    return dx, dxe, dw, (k + min(n, 4096) * E) * (mag * np.abs(xh)).sum((0, 1, 2))


def clip(tensors, limit):
    """(norm, scaled tensors)."""
    norm = math.sqrt(math.fsum(float((np.asarray(x, np.float64) ** 2).sum()) for x in tensors))
    by = limit / norm if math.isfinite(norm) and norm > limit else 1.0
    return norm, [np.asarray(x, np.float64) * by for x in tensors]
