"""Refusals of the gated recurrence, the head norm with rotation and the clipping that need no GPU: the C entry points'
argument checks (fake, never dereferenced pointers) and the Python checks."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p
A, W = 0x10000, 0x20000  # aligned fake pointers
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from sequential_rnn_gb300 import _lib, build
    build.build()
    return _lib.load()


def gdesc(**kw):
    from sequential_rnn_gb300._lib import rnn_gated_desc_t
    d = dict(dtype=1, T=8, B=2, NH=2, D=64, gates=2, flags=0)
    d.update(kw)
    return rnn_gated_desc_t(**d)


def gated(lib, call, desc=None, n_slots=2, nbytes=256, ws=W, **ptr):
    d = ctypes.byref(desc or gdesc(T=1 if call == "step" else 8))
    names = {"fwd": ("Wx", "lens", "s0", "y", "sT", "stash"),
             "bwd": ("Wx", "lens", "stash", "dy", "dsT", "dWx", "ds0"), "step": ("Wx", "slots", "state", "y")}[call]
    p = dict(dict.fromkeys(names, A), lens=0, s0=0, dsT=0, slots=0)
    p.update(ptr)
    a = [P(p[n]) for n in names]
    if call == "step":
        a.insert(2, n_slots)
    else:
        a += [P(ws), nbytes]
    return getattr(lib, "rnn_gated_" + call)(d, *a, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), 1), (dict(T=-1), 1), (dict(B=-1), 1), (dict(NH=-1), 1), (dict(D=0), 1), (dict(gates=1), 1),
    (dict(gates=5), 1), (dict(flags=1), 1), (dict(T=(1 << 30) + 1), 2), (dict(NH=1 << 20, D=1 << 11), 2),
    (dict(B=1 << 24, NH=16, D=64), 2),
])
def test_gated_descriptors(lib, kw, status):
    for call in ("fwd", "bwd", "step"):
        assert gated(lib, call, gdesc(**kw)) == status
    assert lib.rnn_gated_stash_size(ctypes.byref(gdesc(**kw))) == 0


def test_gated_null_and_misaligned(lib):
    for call, need in (("fwd", ("Wx", "y")), ("bwd", ("Wx", "stash", "dy", "dWx")), ("step", ("Wx", "state", "y"))):
        for n in need:
            assert gated(lib, call, **{n: 0}) == 1, (call, n)
            assert gated(lib, call, **{n: A + 1}) == 3, (call, n)
    for n in ("lens", "s0", "sT", "stash"):
        assert gated(lib, "fwd", **{n: A + 2}) == 3
    for n in ("lens", "dsT", "ds0"):
        assert gated(lib, "bwd", **{n: A + 2}) == 3
    assert gated(lib, "fwd", gdesc(dtype=0), Wx=A + 2) == 3
    assert gated(lib, "step", slots=A + 2) == 3
    assert gated(lib, "step", gdesc(T=2)) == gated(lib, "step", n_slots=1) == gated(lib, "step", n_slots=-1) == 1
    assert gated(lib, "step", gdesc(T=1, flags=1 << 30)) == 1
    for call in ("fwd", "bwd"):
        assert gated(lib, call, ws=0) == gated(lib, call, nbytes=128) == 1 and gated(lib, call, ws=W + 16) == 3
        assert gated(lib, call, gdesc(B=0), ws=W + 16, Wx=0) == 3  # the status word is still checked
        for kw in (dict(T=31), dict(T=100, D=36), dict(T=100, D=6, dtype=0)):  # sizes whose kernels do not wait
            assert gated(lib, call, gdesc(flags=1 << 30, **kw)) == 2
    assert gated(lib, "step", gdesc(T=1, B=0), Wx=0, y=0) == gated(lib, "step", gdesc(T=1, NH=0), Wx=0) == 0
    assert lib.rnn_gated_stash_size(ctypes.byref(gdesc(T=17, B=3, NH=2, D=5))) == 3 * 3 * 2 * 5 * 4
    assert lib.rnn_gated_stash_size(ctypes.byref(gdesc(T=0))) == 0


def rdesc(**kw):
    from sequential_rnn_gb300._lib import rnn_rotary_desc_t
    d = dict(dtype=1, T=4, B=2, NQ=2, NK=2, D=64, rot=64, eps=1e-6, flags=0)
    d.update(kw)
    return rnn_rotary_desc_t(**d)


RFWD = ("q", "k", "qw", "kw", "freqs", "pos", "qo", "ko")
RBWD = ("q", "k", "qw", "kw", "freqs", "pos", "dqo", "dko", "dq", "dk", "dqw", "dkw")


def rotary(lib, back, desc=None, st=None, nbytes=1 << 24, ws=W, **ptr):
    names = RBWD if back else RFWD
    p = dict(dict.fromkeys(names, A))
    p.update(ptr)
    a = [ctypes.byref(desc or rdesc()), ctypes.byref(st) if st else None, *[P(p[n]) for n in names]]
    return lib.rnn_head_norm_rotary_bwd(*a, P(ws), nbytes, None) if back else lib.rnn_head_norm_rotary(*a, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), 1), (dict(T=-1), 1), (dict(B=-1), 1), (dict(NQ=-1), 1), (dict(NK=-1), 1), (dict(D=0), 1),
    (dict(rot=-2), 1), (dict(rot=66), 1), (dict(eps=-1.0), 1), (dict(eps=NAN), 1), (dict(flags=4), 1),
    (dict(D=65), 2), (dict(rot=31), 2), (dict(D=4098), 2), (dict(T=1 << 16, B=1 << 15), 2),
    (dict(NQ=1 << 20), 2),
])
def test_rotary_descriptors(lib, kw, status):
    assert rotary(lib, False, rdesc(**kw)) == rotary(lib, True, rdesc(**kw)) == status
    assert lib.rnn_head_norm_rotary_bwd_workspace_size(ctypes.byref(rdesc(**kw))) == 0


def test_rotary_null_and_misaligned(lib):
    from sequential_rnn_gb300._lib import rnn_rotary_strides_t
    for n in ("q", "k", "qo", "ko", "qw", "kw", "freqs"):
        assert rotary(lib, False, **{n: 0}) == 1, n
        assert rotary(lib, False, **{n: A + 1}) == 3, n
    for n in ("q", "k", "dqo", "dko", "dq", "dk", "qw", "freqs", "dqw", "dkw"):
        assert rotary(lib, True, **{n: 0}) == 1, n
        assert rotary(lib, True, **{n: A + 1}) == 3, n
    assert rotary(lib, False, rdesc(flags=2), pos=0) == 1
    assert rotary(lib, False, pos=A + 2) == 3 and rotary(lib, False, freqs=A + 4) == 3
    assert rotary(lib, True, ws=0) == rotary(lib, True, nbytes=64) == 1 and rotary(lib, True, ws=W + 64) == 3
    st = rnn_rotary_strides_t()
    st.q[:] = (-1, 0, 0)
    assert rotary(lib, False, st=st) == 1
    assert rotary(lib, False, rdesc(T=0), q=0, k=0, qo=0, ko=0) == 0
    assert rotary(lib, False, rdesc(NQ=0, NK=0), q=0, k=0, qo=0, ko=0) == 0


def clip(lib, tensors, limit=1.0, dtypes=None, sizes=None, ws=W, nbytes=1 << 24, norm=A, n=None):
    k = len(tensors)
    dt = (ctypes.c_int32 * k)(*(dtypes or [0] * k))
    sz = (ctypes.c_int64 * k)(*(sizes or [16] * k))
    at = (P * k)(*tensors)
    return lib.rnn_clip_grad_norm(k if n is None else n, dt, sz, at, limit, P(norm), P(ws), nbytes, None)


def test_clip_refusals(lib):
    assert clip(lib, [A], limit=-1.0) == clip(lib, [A], limit=NAN) == clip(lib, [A], n=-1) == 1
    assert clip(lib, [A], dtypes=[2]) == clip(lib, [A], sizes=[-1]) == clip(lib, [0]) == 1
    assert clip(lib, [A], sizes=[(1 << 40) + 1]) == 2
    assert clip(lib, [A + 2]) == clip(lib, [A], norm=A + 2) == clip(lib, [A], ws=W + 8) == 3
    assert clip(lib, [A], ws=0) == clip(lib, [A], nbytes=8) == 1
    # the same values twice, whole or in part, in any order
    assert clip(lib, [A, A]) == clip(lib, [A, A + 60]) == clip(lib, [A + 60, 4 * A, A]) == 1
    assert clip(lib, [4 * A, A, A + 30], dtypes=[0, 1, 1]) == 1
    assert lib.rnn_clip_grad_norm(1, None, None, None, 1.0, None, P(W), 1 << 20, None) == 1
    assert lib.rnn_clip_grad_norm_workspace_size(-1) == 0 and lib.rnn_clip_grad_norm_workspace_size(0) >= 8


def test_python_refusals():
    import sequential_rnn_gb300 as S
    x = torch.zeros(3, 2, 2, 8)
    for f in (lambda: S.gated_recurrence(x), lambda: S.gated_recurrence_step(x[0], x[0]),
              lambda: S.gated_recurrence_backward(x, x, x), lambda: S.head_norm_rotary(x, x, None, None, None),
              lambda: S.clip_grad_norm([x], 1.0), lambda: S.grad_norm([x])):
        with pytest.raises(ValueError, match="CUDA"):
            f()
    with pytest.raises(TypeError):
        S.gated_recurrence([1.0])
    with pytest.raises(TypeError):
        S.clip_grad_norm([1.0], 1.0)
    with pytest.raises(TypeError):
        S.clip_grad_norm(1.0, 1.0)
    with pytest.raises(ValueError):
        S.rotary_frequencies(7, device="cpu")


def test_rotary_frequencies():
    import sequential_rnn_gb300 as S
    f = S.rotary_frequencies(8, 100.0, device="cpu")
    assert f.dtype == torch.float64 and f.tolist() == pytest.approx([1, 100 ** -0.25, 0.1, 100 ** -0.75])
    assert S.rotary_frequencies(0, device="cpu").numel() == 0
