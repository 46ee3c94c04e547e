"""fp64 oracle of the language-model operators: linear attention with a decay per
head (token by token), the root-mean-square norm with its 8-bit output, and the
projection with a scale for each block of 128.  Test infrastructure (numpy)."""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
BLOCK = 128

__all__ = ["linear_attention", "linear_attention_backward", "linear_attention_bound", "rms_norm",
           "rms_norm_backward", "quantize", "e4m3", "proj_fp8"]


def _lens(T, B, lens):
    return np.full(B, T) if lens is None else np.clip(np.asarray(lens), 0, T)


def linear_attention(q, k, v, log_decay, s0=None, lens=None, scale=1.0):
    """q, k [T,B,NH,Dk], v [T,B,NH,Dv] -> o [T,B,NH,Dv], final state [B,NH,Dk,Dv]."""
    T, B, NH, Dk = q.shape
    Dv = v.shape[-1]
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    lam = np.exp(np.asarray(log_decay, np.float64))
    s = np.zeros((B, NH, Dk, Dv)) if s0 is None else np.array(s0, np.float64)
    o = np.zeros((T, B, NH, Dv))
    for b, n in enumerate(_lens(T, B, lens)):
        for t in range(n):
            s[b] = lam[:, None, None] * s[b] + k[t, b][:, :, None] * v[t, b][:, None, :]
            o[t, b] = scale * np.einsum("hk,hkv->hv", q[t, b], s[b])
    return o, s


def linear_attention_backward(q, k, v, log_decay, do, s0=None, dsT=None, lens=None, scale=1.0):
    """dq, dk, dv and the initial state's gradient of sum(o do) + sum(s_T dsT)."""
    T, B, NH, Dk = q.shape
    Dv = v.shape[-1]
    q, k, v, do = (np.asarray(x, np.float64) for x in (q, k, v, do))
    lam = np.exp(np.asarray(log_decay, np.float64))[:, None, None]
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    s = np.zeros((B, NH, Dk, Dv)) if s0 is None else np.array(s0, np.float64)
    ds = np.zeros((B, NH, Dk, Dv)) if dsT is None else np.array(dsT, np.float64)
    for b, n in enumerate(_lens(T, B, lens)):
        for t in range(n):
            s[b] = lam * s[b] + k[t, b][:, :, None] * v[t, b][:, None, :]
            dq[t, b] = scale * np.einsum("hkv,hv->hk", s[b], do[t, b])
        for t in reversed(range(n)):
            ds[b] += scale * q[t, b][:, :, None] * do[t, b][:, None, :]
            dk[t, b] = np.einsum("hkv,hv->hk", ds[b], v[t, b])
            dv[t, b] = np.einsum("hkv,hk->hv", ds[b], k[t, b])
            ds[b] *= lam
    return dq, dk, dv, ds


def linear_attention_bound(x, a, c, log_decay, s0=None, lens=None, reverse=False, intra=1.0,
                           inter=1.0, upd=1.0, chunk=64):
    """Sums of magnitudes that bound what rounding can change in a chunked pass:
    ((rounded, all), state).  rounded: per output sum_j |score_j c_j| inside the token's chunk
    + |x| |S| with the state S at the chunk's start, what rounding the scores and the state as operands
    is relative to.  all, state: the magnitudes of all products behind an output and
    behind the final state, what the error of their fp32 sums is relative to.  (x, a, c) is
    (q, k, v), or what takes their places in a gradient."""
    T, B, NH, D = x.shape
    E = c.shape[-1]
    x, a, c = (np.asarray(t, np.float64) for t in (x, a, c))
    lam = np.exp(np.asarray(log_decay, np.float64))
    mag, full = np.zeros((T, B, NH, E)), np.zeros((T, B, NH, E))
    fin = np.zeros((B, NH, D, E))
    for b, n in enumerate(_lens(T, B, lens)):
        at = np.arange(n)[::-1] if reverse else np.arange(n)
        sh = 1 if reverse else 0
        s = np.zeros((NH, D, E)) if s0 is None else np.array(s0[b], np.float64)
        m = np.abs(s)
        for lo in range(0, n, chunk):
            i = at[lo:lo + chunk]
            xs, as_, cs = (t[i, b] for t in (x, a, c))        # [C, NH, *]
            C = len(i)
            p = np.arange(C)
            d = np.where(p[:, None] >= p[None], lam[:, None, None] ** np.maximum(p[:, None] - p[None], 0), 0)
            sc = np.abs(np.einsum("ihd,jhd->hij", xs, as_) * d * intra)
            w = lam[None] ** (p[:, None] + 1 - sh)
            mag[i, b] = (np.einsum("hij,jhe->ihe", sc, np.abs(cs))
                         + np.abs(inter) * w[..., None] * np.einsum("ihd,hde->ihe", np.abs(xs), np.abs(s)))
            sa = np.einsum("ihd,jhd->hij", np.abs(xs), np.abs(as_)) * np.abs(d * intra)
            full[i, b] = (np.einsum("hij,jhe->ihe", sa, np.abs(cs))
                          + np.abs(inter) * w[..., None] * np.einsum("ihd,hde->ihe", np.abs(xs), m))
            wj = upd * lam[None] ** (C - 1 - p[:, None] + sh)
            s = (lam ** C)[:, None, None] * s + np.einsum("jhd,jhe,jh->hde", as_, cs, wj)
            m = (lam ** C)[:, None, None] * m + np.einsum("jhd,jhe,jh->hde", np.abs(as_), np.abs(cs), np.abs(wj))
        fin[b] = m
    return (mag, full), fin


def e4m3(x):
    """x rounded to the nearest e4m3 value (ties to even), magnitudes over 448 to 448."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), E4M3_MAX)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    step = 2.0 ** (e - 3)
    return np.sign(x) * np.minimum(np.round(a / step) * step, E4M3_MAX)


def quantize(y, rows=1):
    """(values, scales) of y [M, K] with one scale for each block of `rows` x 128."""
    M, K = y.shape
    mb, kb = -(-M // rows), -(-K // BLOCK)
    s = np.ones((mb, kb))
    q = np.zeros((M, K))
    for i in range(mb):
        for j in range(kb):
            part = np.asarray(y[i * rows:(i + 1) * rows, j * BLOCK:(j + 1) * BLOCK], np.float64)
            top = np.abs(part).max()
            if top > 0:
                s[i, j] = top / E4M3_MAX
            q[i * rows:(i + 1) * rows, j * BLOCK:(j + 1) * BLOCK] = e4m3(part / s[i, j])
    return q, s


def rms_norm(h, w, eps):
    """(y, rstd) of rows h [R, N]."""
    h = np.asarray(h, np.float64)
    r = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h * r[:, None] * np.asarray(w, np.float64), r


def rms_norm_backward(dy, h, w, rstd, dh=None):
    dy, h, w, r = (np.asarray(t, np.float64) for t in (dy, h, w, rstd))
    xh = h * r[:, None]
    g = dy * w
    dx = r[:, None] * (g - xh * (g * xh).mean(1, keepdims=True))
    if dh is not None:
        dx = dx + np.asarray(dh, np.float64)
    return dx, (dy * xh).sum(0)


def proj_fp8(xq, xs, wq, ws, bias=None):
    """(y, sum of magnitudes) of the scaled product."""
    M, K = xq.shape
    N = wq.shape[0]
    x = np.asarray(xq, np.float64) * np.repeat(np.asarray(xs, np.float64), BLOCK, 1)[:, :K]
    w = np.asarray(wq, np.float64) * np.repeat(np.repeat(np.asarray(ws, np.float64), BLOCK, 0)[:N], BLOCK, 1)[:, :K]
    b = 0.0 if bias is None else np.asarray(bias, np.float64)[None]
    return x @ w.T + b, np.abs(x) @ np.abs(w).T + np.abs(b)
