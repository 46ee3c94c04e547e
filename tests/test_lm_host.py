"""Refusals of the language-model operators that need no GPU: the C entry points'
argument checks (fake, never dereferenced pointers) and the Python checks."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p
A, W = 0x10000, 0x20000  # aligned fake pointers


@pytest.fixture(scope="module")
def lib():
    from sequential_rnn_gb300 import _lib, build
    build.build()
    return _lib.load()


def norm(lib, dtype=1, rows=4, N=64, eps=1e-6, x=A, res=A, w=A, h=A, y=A, scale=None, rstd=None):
    return lib.rnn_rms_norm(dtype, rows, N, eps, P(x), P(res), P(w), P(h), P(y), P(scale), P(rstd), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), 1), (dict(rows=-1), 1), (dict(N=0), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(x=0), 1), (dict(w=0), 1), (dict(y=0), 1), (dict(x=A + 1), 3),
    (dict(dtype=0, res=A + 2), 3), (dict(w=A + 2), 3), (dict(scale=A + 2), 3), (dict(rstd=A + 1), 3),
    (dict(h=A + 1), 3), (dict(rows=0, x=0, y=0, w=0), 0),
])
def test_rms_norm_refusals(lib, kw, status):
    assert norm(lib, **kw) == status


def norm_bwd(lib, dtype=1, rows=4, N=64, dy=A, h=A, w=A, rstd=A, dh=A, dx=A, dw=A, ws=A, nbytes=1 << 20):
    return lib.rnn_rms_norm_bwd(dtype, rows, N, P(dy), P(h), P(w), P(rstd), P(dh), P(dx), P(dw), P(ws),
                                nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=9), 1), (dict(rows=-1), 1), (dict(N=-3), 1), (dict(dy=0), 1), (dict(h=0), 1),
    (dict(rstd=0), 1), (dict(dx=0), 1), (dict(w=0), 1), (dict(ws=0), 1), (dict(nbytes=64), 1),
    (dict(ws=A + 64), 3), (dict(dy=A + 1), 3), (dict(dw=A + 2), 3), (dict(dh=A + 1), 3),
    (dict(rows=0, dw=0), 0),
])
def test_rms_norm_bwd_refusals(lib, kw, status):
    assert norm_bwd(lib, **kw) == status


def test_rms_norm_bwd_workspace(lib):
    f = lib.rnn_rms_norm_bwd_workspace_size
    assert f(-1, 8) == 0 and f(8, 0) == 0 and f(0, 8) >= 256 and f(5, 100) >= 256 + 5 * 100 * 4


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), 1), (dict(N=0), 1), (dict(K=0), 1), (dict(W=0), 1), (dict(Wq=0), 1), (dict(Ws=0), 1),
    (dict(W=A + 1), 3), (dict(Ws=A + 2), 3), (dict(N=65536 * 128), 2),
])
def test_quantize_weight_refusals(lib, kw, status):
    a = dict(dtype=1, N=8, K=16, W=A, Wq=A, Ws=A)
    a.update(kw)
    assert lib.rnn_quantize_weight(a["dtype"], a["N"], a["K"], P(a["W"]), P(a["Wq"]), P(a["Ws"]), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), 1), (dict(N=0), 1), (dict(K=0), 1), (dict(K=24), 2), (dict(N=12), 2),
    (dict(M=65535 * 128 + 1), 2), (dict(xq=0), 1), (dict(xs=0), 1), (dict(Wq=0), 1), (dict(Ws=0), 1),
    (dict(y=0), 1), (dict(ws=0), 1), (dict(nbytes=128), 1), (dict(ws=A + 16), 3), (dict(xq=A + 8), 3),
    (dict(Wq=A + 8), 3), (dict(y=A + 2), 3), (dict(xs=A + 2), 3), (dict(bias=A + 1), 3),
])
def test_input_proj_fp8_refusals(lib, kw, status):
    a = dict(M=4, N=16, K=32, xq=A, xs=A, Wq=A, Ws=A, bias=0, y=A, ws=W, nbytes=256)
    a.update(kw)
    assert lib.rnn_input_proj_fp8(a["M"], a["N"], a["K"], P(a["xq"]), P(a["xs"]), P(a["Wq"]), P(a["Ws"]),
                                  P(a["bias"]), P(a["y"]), P(a["ws"]), a["nbytes"], None) == status


def ldesc(**kw):
    from sequential_rnn_gb300._lib import rnn_linattn_desc_t
    d = dict(dtype=1, T=8, B=2, NH=2, Dk=64, Dv=64, scale=1.0, flags=0)
    d.update(kw)
    return rnn_linattn_desc_t(**d)


BAD_DESC = [(dict(dtype=2), 1), (dict(T=-1), 1), (dict(B=-1), 1), (dict(NH=-1), 1), (dict(Dk=0), 1),
            (dict(flags=1), 1), (dict(Dk=48), 2), (dict(Dv=512), 2), (dict(T=(1 << 30) + 1), 2),
            (dict(B=1 << 20, NH=2), 2)]


def strides(**kw):
    from sequential_rnn_gb300._lib import rnn_linattn_strides_t
    s = rnn_linattn_strides_t()
    for n in ("q", "k", "v", "o"):
        getattr(s, n)[:] = kw.get(n, (256, 128, 64))
    return s


def fwd(lib, desc=None, st=None, nbytes=1 << 30, **ptr):
    p = dict(q=A, k=A, v=A, g=A, lens=0, s0=0, o=A, sT=0, ws=W)
    p.update(ptr)
    return lib.rnn_linattn_fwd(ctypes.byref(desc or ldesc()), ctypes.byref(st) if st else None,
                               *[P(p[n]) for n in ("q", "k", "v", "g", "lens", "s0", "o", "sT", "ws")],
                               nbytes, None)


def bwd(lib, desc=None, st=None, nbytes=1 << 30, **ptr):
    names = ("q", "k", "v", "g", "lens", "s0", "do", "dsT", "dq", "dk", "dv", "ds0", "ws")
    p = dict(dict.fromkeys(names, A), lens=0, s0=0, dsT=0, ds0=0, ws=W)
    p.update(ptr)
    return lib.rnn_linattn_bwd(ctypes.byref(desc or ldesc()), ctypes.byref(st) if st else None,
                               *[P(p[n]) for n in names], nbytes, None)


def step(lib, desc=None, st=None, n_slots=2, **ptr):
    p = dict(q=A, k=A, v=A, g=A, slots=0, state=A, o=A)
    p.update(ptr)
    return lib.rnn_linattn_step(ctypes.byref(desc or ldesc(T=1)), ctypes.byref(st) if st else None,
                                *[P(p[n]) for n in ("q", "k", "v", "g", "slots")], n_slots,
                                P(p["state"]), P(p["o"]), None)


@pytest.mark.parametrize("kw,status", BAD_DESC)
def test_linattn_descriptors(lib, kw, status):
    d = ldesc(**kw)
    assert fwd(lib, d) == bwd(lib, d) == step(lib, d) == status
    assert lib.rnn_linattn_workspace_size(ctypes.byref(d), 0) == 0


def test_linattn_null_and_misaligned(lib):
    for n in ("q", "k", "v", "g", "o", "ws"):
        assert fwd(lib, **{n: 0}) == 1, n
    for n in ("q", "k", "v", "g", "do", "dq", "dk", "dv", "ws"):
        assert bwd(lib, **{n: 0}) == 1, n
    for n in ("q", "k", "v", "g", "o", "state"):
        assert step(lib, **{n: 0}) == 1, n
    for n in ("q", "v", "o", "s0", "sT"):
        assert fwd(lib, **{n: A + 8}) == 3, n
    for n in ("do", "dq", "dsT", "ds0"):
        assert bwd(lib, **{n: A + 8}) == 3, n
    assert fwd(lib, lens=A + 2) == fwd(lib, ws=W + 16) == step(lib, state=A + 4) == 3
    assert fwd(lib, nbytes=8) == bwd(lib, nbytes=8) == 1
    assert fwd(lib, st=strides(k=(256, 128, 60))) == 3
    assert fwd(lib, st=strides(q=(-256, 128, 64))) == 3
    assert step(lib, st=strides(v=(0, 128, 36))) == 3
    assert bwd(lib, dsT=A, ds0=A) == 1          # read by one pass, written by another
    assert step(lib, ldesc(T=2)) == 1 and step(lib, n_slots=1) == 1 and step(lib, n_slots=-1) == 1
    assert lib.rnn_linattn_workspace_size(ctypes.byref(ldesc()), 2) == 0
    assert fwd(lib, ldesc(B=0), q=0, k=0, v=0, o=0, g=0, ws=W + 1) == 3  # the status word is still checked


def test_python_refusals():
    import sequential_rnn_gb300 as S
    x, w = torch.zeros(2, 8), torch.zeros(8)
    with pytest.raises(ValueError):
        S.rms_norm(x, w)                         # not on a CUDA device
    with pytest.raises(TypeError):
        S.rms_norm([1.0], w)
    with pytest.raises(ValueError):
        S.quantize_weight(x)
    with pytest.raises(ValueError):
        S.input_proj_fp8(x, x, x, x)
    q = torch.zeros(3, 1, 2, 32)
    for f in (S.linear_attention, S.linear_attention_step):
        with pytest.raises((ValueError, TypeError)):
            f(q, q, q, torch.zeros(2), None) if f is S.linear_attention_step else f(q, q, q, torch.zeros(2))
