"""Operators of language models around and beside the recurrences.

``rms_norm`` / ``rms_norm_backward``   root-mean-square norm with the residual's
                                       addition, output in the input type or in
                                       8 bits with a scale for each 128 columns
``quantize_weight``, ``input_proj_fp8`` the input projection in 8-bit floating
                                       point with a scale for each block of 128
``linear_attention`` (``_backward``, ``_step``)
                                       matrix-memory recurrence with a decay for
                                       each head: prompts, gradient, single tokens

As in the package's top level, the functions named like the C entry points only
marshal arguments, and the others check them, allocate the outputs and raise
``RnnError`` on a non-OK status.  Everything runs on ``stream`` (a
``torch.cuda.Stream`` or a raw handle; None: the current stream), outputs and
workspace are allocated for that stream, and inputs made on another one have to
be ordered before it by the caller.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib
from ._lib import RNN_BF16, RNN_F32, rnn_linattn_desc_t, rnn_linattn_strides_t

__all__ = ["rnn_rms_norm", "rnn_rms_norm_bwd_workspace_size", "rnn_rms_norm_bwd",
           "rnn_quantize_weight", "rnn_input_proj_fp8", "rnn_linattn_workspace_size",
           "rnn_linattn_fwd", "rnn_linattn_bwd", "rnn_linattn_step", "rms_norm",
           "rms_norm_backward", "quantize_weight", "input_proj_fp8", "linear_attention",
           "linear_attention_backward", "linear_attention_step"]

_DT = {torch.float32: RNN_F32, torch.bfloat16: RNN_BF16}
_E4M3 = torch.float8_e4m3fn
BLOCK = 128  # columns (and weight rows) that share a scale


def _raise(status, where):
    from . import RnnError
    raise RnnError(status, where)


def _at(t):
    return t.data_ptr() if t is not None else None


def _want(name, t, shape, dtype, device, contiguous=True):
    # one condition first: these calls take microseconds, and so do the kernels of a single token
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device
            and (not contiguous or t.is_contiguous())):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name}: expected a tensor on {device}, got {t.device}")
    raise ValueError(f"{name}: tensor must be contiguous")


def _device(name, t):
    """The CUDA device of the leading operand, which has to be the current one."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: tensor must live on a CUDA device")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name}: tensor must live on the current CUDA device")
    return t.device


def _dtype(name, t):
    if t.dtype not in _DT:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    return t.dtype


def _handle(stream):
    """The raw handle of a stream; None: the current one."""
    if stream is None:
        return _current(torch.cuda.current_device())
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


# (torch.cuda.current_stream() makes a Stream object: 3 us against 0.1 us)
_current = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _for_stream(f):
    """Runs f, which works on the current stream, on the stream that its caller names: what f
    allocates then belongs to that stream, too."""
    @functools.wraps(f)
    def call(*args, stream=None, **kw):
        if stream is None:
            return f(*args, **kw)
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream))
        with torch.cuda.stream(stream):
            return f(*args, **kw)
    return call


def _read(ws, where):
    from . import rnn_read_status
    st = rnn_read_status(ws)
    if st:
        _raise(st, where + " (device)")


# ------------------------------------------------------ C-named wrappers --
def rnn_rms_norm(dtype, rows, N, eps, x, residual, weight, h, y, scale, rstd, stream=None) -> int:
    return _lib.load().rnn_rms_norm(dtype, rows, N, eps, _at(x), _at(residual), _at(weight), _at(h),
                                    _at(y), _at(scale), _at(rstd), _handle(stream))


def rnn_rms_norm_bwd_workspace_size(rows, N) -> int:
    return int(_lib.load().rnn_rms_norm_bwd_workspace_size(rows, N))


def rnn_rms_norm_bwd(dtype, rows, N, dy, h, weight, rstd, dh, dx, dw, workspace, stream=None) -> int:
    return _lib.load().rnn_rms_norm_bwd(dtype, rows, N, _at(dy), _at(h), _at(weight), _at(rstd),
                                        _at(dh), _at(dx), _at(dw), _at(workspace),
                                        workspace.nbytes if workspace is not None else 0,
                                        _handle(stream))


def rnn_quantize_weight(dtype, N, K, W, Wq, Ws, stream=None) -> int:
    return _lib.load().rnn_quantize_weight(dtype, N, K, _at(W), _at(Wq), _at(Ws), _handle(stream))


def rnn_input_proj_fp8(M, N, K, xq, xs, Wq, Ws, bias, y, workspace, stream=None) -> int:
    return _lib.load().rnn_input_proj_fp8(M, N, K, _at(xq), _at(xs), _at(Wq), _at(Ws), _at(bias),
                                          _at(y), _at(workspace),
                                          workspace.nbytes if workspace is not None else 0,
                                          _handle(stream))


def rnn_linattn_workspace_size(desc, pass_=0) -> int:
    return int(_lib.load().rnn_linattn_workspace_size(ctypes.byref(desc), pass_))


def _sref(strides):
    return ctypes.byref(strides) if strides is not None else None


def rnn_linattn_fwd(desc, strides, q, k, v, log_decay, lens, state0, o, stateT, workspace,
                    stream=None) -> int:
    return _lib.load().rnn_linattn_fwd(ctypes.byref(desc), _sref(strides), _at(q), _at(k), _at(v),
                                       _at(log_decay), _at(lens), _at(state0), _at(o), _at(stateT),
                                       _at(workspace), workspace.nbytes if workspace is not None else 0,
                                       _handle(stream))


def rnn_linattn_bwd(desc, strides, q, k, v, log_decay, lens, state0, do, dstateT, dq, dk, dv,
                    dstate0, workspace, stream=None) -> int:
    return _lib.load().rnn_linattn_bwd(ctypes.byref(desc), _sref(strides), _at(q), _at(k), _at(v),
                                       _at(log_decay), _at(lens), _at(state0), _at(do), _at(dstateT),
                                       _at(dq), _at(dk), _at(dv), _at(dstate0), _at(workspace),
                                       workspace.nbytes if workspace is not None else 0,
                                       _handle(stream))


def rnn_linattn_step(desc, strides, q, k, v, log_decay, slots, n_slots, state, o, stream=None) -> int:
    return _lib.load().rnn_linattn_step(ctypes.byref(desc), _sref(strides), _at(q), _at(k), _at(v),
                                        _at(log_decay), _at(slots), n_slots, _at(state), _at(o),
                                        _handle(stream))


# ------------------------------------------------------------------ norm --
@_for_stream
def rms_norm(x, weight, residual=None, *, eps=1e-6, quantize=False, train=False):
    """h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight over the last dimension.

    x, residual [..., N] bf16 or fp32, weight [N] fp32.  Returns ``h`` (x itself
    without a residual), ``y`` (x's type; with ``quantize`` e4m3, and ``scale``
    [..., ceil(N/128)] fp32) and with ``train`` the ``rstd`` [...] fp32 that
    ``rms_norm_backward`` takes.
    """
    dev, dt = _device("x", x), _dtype("x", x)
    shape = x.shape
    if not shape:
        raise ValueError("x: expected at least one dimension")
    N = shape[-1]
    _want("x", x, shape, dt, dev)
    _want("weight", weight, (N,), torch.float32, dev)
    if residual is not None:
        _want("residual", residual, shape, dt, dev)
    h = torch.empty_like(x) if residual is not None else None
    out = {"h": x if h is None else h}
    scale = rstd = None
    if quantize:
        y = torch.empty(shape, dtype=_E4M3, device=dev)
        scale = out["scale"] = torch.empty(shape[:-1] + (-(-N // BLOCK),), dtype=torch.float32,
                                           device=dev)
    else:
        y = torch.empty_like(x)
    if train:
        rstd = out["rstd"] = torch.empty(shape[:-1], dtype=torch.float32, device=dev)
    out["y"] = y
    st = _lib.load().rnn_rms_norm(_DT[dt], x.numel() // N if N else 0, N, eps, x.data_ptr(),
                                  _at(residual), weight.data_ptr(), _at(h), y.data_ptr(), _at(scale),
                                  _at(rstd), _handle(None))
    if st:
        _raise(st, "rnn_rms_norm")
    return out


@_for_stream
def rms_norm_backward(dy, h, weight, rstd, *, dh=None):
    """Gradient of ``rms_norm`` from its ``h`` and ``rstd``: ``dx`` (the gradient of x
    and of the residual, ``dh`` included) and ``dw`` [N] fp32."""
    dev, dt = _device("h", h), _dtype("h", h)
    shape = h.shape
    if not shape:
        raise ValueError("h: expected at least one dimension")
    N = shape[-1]
    _want("h", h, shape, dt, dev)
    _want("dy", dy, shape, dt, dev)
    _want("weight", weight, (N,), torch.float32, dev)
    _want("rstd", rstd, shape[:-1], torch.float32, dev)
    if dh is not None:
        _want("dh", dh, shape, dt, dev)
    lib = _lib.load()
    rows = h.numel() // N if N else 0
    nbytes = lib.rnn_rms_norm_bwd_workspace_size(rows, N)
    dx = torch.empty_like(h)
    dw = torch.empty(N, dtype=torch.float32, device=dev)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    st = lib.rnn_rms_norm_bwd(_DT[dt], rows, N, dy.data_ptr(), h.data_ptr(), weight.data_ptr(),
                              rstd.data_ptr(), _at(dh), dx.data_ptr(), dw.data_ptr(), ws.data_ptr(),
                              nbytes, _handle(None))
    if st:
        _raise(st, "rnn_rms_norm_bwd")
    return {"dx": dx, "dw": dw}


# ------------------------------------------------------------ projection --
@_for_stream
def quantize_weight(W):
    """W [N, K] (bf16 or fp32) as e4m3 [N, K] and a scale for each 128 x 128 block."""
    dev, dt = _device("W", W), _dtype("W", W)
    if W.dim() != 2:
        raise ValueError("W: expected [N, K]")
    N, K = W.shape
    _want("W", W, (N, K), dt, dev)
    Wq = torch.empty((N, K), dtype=_E4M3, device=dev)
    Ws = torch.empty((-(-N // BLOCK), -(-K // BLOCK)), dtype=torch.float32, device=dev)
    st = _lib.load().rnn_quantize_weight(_DT[dt], N, K, W.data_ptr(), Wq.data_ptr(), Ws.data_ptr(),
                                         _handle(None))
    if st:
        _raise(st, "rnn_quantize_weight")
    return Wq, Ws


@_for_stream
def input_proj_fp8(xq, xs, Wq, Ws, bias=None, *, check=True):
    """Wx = x W^T + bias from 8-bit operands through rnn_input_proj_fp8.

    xq [..., K], Wq [N, K] e4m3; xs [..., ceil(K/128)], Ws [ceil(N/128), ceil(K/128)]
    fp32 (``rms_norm(quantize=True)``'s and ``quantize_weight``'s); bias [N] fp32 or
    None -> [..., N] bf16, as ``input_proj`` gives it.
    """
    dev = _device("xq", xq)
    if xq.dim() < 1 or not isinstance(Wq, torch.Tensor) or Wq.dim() != 2:
        raise ValueError("expected xq [..., K] and Wq [N, K]")
    lead, K, N = xq.shape[:-1], xq.shape[-1], Wq.shape[0]
    kb = -(-K // BLOCK)
    _want("xq", xq, xq.shape, _E4M3, dev)
    _want("xs", xs, lead + (kb,), torch.float32, dev)
    _want("Wq", Wq, (N, K), _E4M3, dev)
    _want("Ws", Ws, (-(-N // BLOCK), kb), torch.float32, dev)
    if bias is not None:
        _want("bias", bias, (N,), torch.float32, dev)
    y = torch.empty(lead + (N,), dtype=torch.bfloat16, device=dev)
    ws = torch.empty(256, dtype=torch.uint8, device=dev)
    st = _lib.load().rnn_input_proj_fp8(xq.numel() // K if K else 0, N, K, xq.data_ptr(),
                                        xs.data_ptr(), Wq.data_ptr(), Ws.data_ptr(), _at(bias),
                                        y.data_ptr(), ws.data_ptr(), 256, _handle(None))
    if st:
        _raise(st, "rnn_input_proj_fp8")
    if check:
        _read(ws, "rnn_input_proj_fp8")
    return y


# ------------------------------------------------------ linear attention --
@functools.lru_cache(maxsize=256)
def _desc(dtype, T, B, NH, Dk, Dv, scale):
    """A descriptor with its workspace sizes (forward, backward); read only."""
    desc = rnn_linattn_desc_t(dtype, T, B, NH, Dk, Dv, scale, 0)
    return desc, *(max(rnn_linattn_workspace_size(desc, i), 256) for i in (0, 1))


@functools.lru_cache(maxsize=256)
def _strides(q, k, v, o):
    st = rnn_linattn_strides_t()
    st.q[:], st.k[:], st.v[:], st.o[:] = q, k, v, o
    return st


def _stride_of(name, t):
    *s, last = t.stride()
    if last != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    # (a dimension of one element has no stride to speak of)
    s = [x if n > 1 else 0 for x, n in zip(s, t.shape)]
    return (*[0] * (3 - len(s)), *s)


def _linattn(q, k, v, log_decay, scale, lead, do=None):
    """Checks the operands with `lead` dimensions before the heads'; (desc, workspace bytes forward and
    backward, strides, device, dtype)."""
    dev, dt = _device("q", q), _dtype("q", q)
    if q.dim() != lead + 2 or not isinstance(v, torch.Tensor) or v.dim() != lead + 2:
        raise ValueError("expected q, k, v of shape " + ("[T, B, NH, D]" if lead == 2 else "[B, NH, D]"))
    shape = q.shape
    *lead_shape, NH, Dk = shape
    Dv = v.shape[-1]
    _want("k", k, shape, dt, dev, False)
    _want("v", v, (*lead_shape, NH, Dv), dt, dev, False)
    _want("log_decay", log_decay, (NH,), torch.float32, dev)
    T, B = lead_shape if lead == 2 else (1, lead_shape[0])
    if do is not None:
        _want("do", do, (T, B, NH, Dv), dt, dev, False)
    st = None
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous()
            and (do is None or do.is_contiguous())):
        st = _strides(_stride_of("q", q), _stride_of("k", k), _stride_of("v", v),
                      _stride_of("do", do) if do is not None else (B * NH * Dv, NH * Dv, Dv))
    return *_desc(_DT[dt], T, B, NH, Dk, Dv, max(Dk, 1) ** -0.5 if scale is None else scale), st, dev, dt


@_for_stream
def linear_attention(q, k, v, log_decay, *, state=None, lens=None, scale=None, check=True):
    """S_t = exp(log_decay) S_{t-1} + k_t v_t^T, o_t = scale q_t S_t through rnn_linattn_fwd.

    q, k [T, B, NH, Dk], v [T, B, NH, Dv] bf16 or fp32 (strided views with a
    contiguous last dimension are taken as they are), log_decay [NH] fp32,
    state [B, NH, Dk, Dv] fp32 or None, lens [B] int32 or None (tokens of each row
    that count), scale Dk^-0.5 unless given.  Returns ``o`` [T, B, NH, Dv], ``state``
    (after the last token) and the ``workspace``.
    """
    desc, nbytes, _, st, dev, dt = _linattn(q, k, v, log_decay, scale, 2)
    T, B, NH, Dk, Dv = desc.T, desc.B, desc.NH, desc.Dk, desc.Dv
    if state is not None:
        _want("state", state, (B, NH, Dk, Dv), torch.float32, dev)
    if lens is not None:
        _want("lens", lens, (B,), torch.int32, dev)
    lib = _lib.load()
    o = torch.empty((T, B, NH, Dv), dtype=dt, device=dev)
    fin = torch.empty((B, NH, Dk, Dv), dtype=torch.float32, device=dev)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    e = lib.rnn_linattn_fwd(ctypes.byref(desc), _sref(st), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                            log_decay.data_ptr(), _at(lens), _at(state), o.data_ptr(), fin.data_ptr(),
                            ws.data_ptr(), nbytes, _handle(None))
    if e:
        _raise(e, "rnn_linattn_fwd")
    if check:
        _read(ws, "rnn_linattn_fwd")
    return {"o": o, "state": fin, "workspace": ws}


@_for_stream
def linear_attention_backward(q, k, v, log_decay, do, *, state=None, dstate=None, lens=None,
                              scale=None, check=True):
    """Gradients of ``linear_attention`` from its inputs, ``do`` [T, B, NH, Dv] (may be
    strided as they may) and ``dstate`` (of the final state, or None): ``dq``, ``dk``,
    ``dv`` and ``dstate`` (of the initial state)."""
    if not isinstance(do, torch.Tensor):
        raise TypeError("do: expected a torch.Tensor")
    desc, _, nbytes, st, dev, dt = _linattn(q, k, v, log_decay, scale, 2, do)
    T, B, NH, Dk, Dv = desc.T, desc.B, desc.NH, desc.Dk, desc.Dv
    for name, t in (("state", state), ("dstate", dstate)):
        if t is not None:
            _want(name, t, (B, NH, Dk, Dv), torch.float32, dev)
    if lens is not None:
        _want("lens", lens, (B,), torch.int32, dev)
    lib = _lib.load()
    dq = torch.empty((T, B, NH, Dk), dtype=dt, device=dev)
    dk, dv = torch.empty_like(dq), torch.empty((T, B, NH, Dv), dtype=dt, device=dev)
    ds0 = torch.empty((B, NH, Dk, Dv), dtype=torch.float32, device=dev)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    e = lib.rnn_linattn_bwd(ctypes.byref(desc), _sref(st), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                            log_decay.data_ptr(), _at(lens), _at(state), do.data_ptr(), _at(dstate),
                            dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ds0.data_ptr(),
                            ws.data_ptr(), nbytes, _handle(None))
    if e:
        _raise(e, "rnn_linattn_bwd")
    if check:
        _read(ws, "rnn_linattn_bwd")
    return {"dq": dq, "dk": dk, "dv": dv, "dstate": ds0, "workspace": ws}


@_for_stream
def linear_attention_step(q, k, v, log_decay, state, *, slots=None, scale=None):
    """One token for each row: q, k [B, NH, Dk], v [B, NH, Dv] against the cache ``state``
    [n_slots, NH, Dk, Dv] fp32, updated in place; row b uses state slots[b] (int32; None:
    state b).  A slot outside the cache gives zeros; no two rows may name the same one.
    Returns o [B, NH, Dv]."""
    desc, _, _, st, dev, dt = _linattn(q, k, v, log_decay, scale, 1)
    B, NH, Dk, Dv = desc.B, desc.NH, desc.Dk, desc.Dv
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state: expected [n_slots, NH, Dk, Dv]")
    _want("state", state, (state.shape[0], NH, Dk, Dv), torch.float32, dev)
    if slots is not None:
        _want("slots", slots, (B,), torch.int32, dev)
    o = torch.empty((B, NH, Dv), dtype=dt, device=dev)
    e = _lib.load().rnn_linattn_step(ctypes.byref(desc), _sref(st), q.data_ptr(), k.data_ptr(),
                                     v.data_ptr(), log_decay.data_ptr(), _at(slots), state.shape[0],
                                     state.data_ptr(), o.data_ptr(), _handle(None))
    if e:
        _raise(e, "rnn_linattn_step")
    return o
