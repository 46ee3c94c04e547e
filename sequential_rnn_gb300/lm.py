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
marshal arguments, and the others check them, allocate the outputs (both in
csrc/binding.cpp) and raise ``RnnError`` on a non-OK status.  Everything runs on ``stream`` (a
``torch.cuda.Stream`` or a raw handle; None: the current stream), outputs and
workspace are allocated for that stream, and inputs made on another one have to
be ordered before it, and kept until it is done with them, by the caller.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib

__all__ = ["rnn_rms_norm", "rnn_rms_norm_bwd_workspace_size", "rnn_rms_norm_bwd",
           "rnn_quantize_weight", "rnn_input_proj_fp8", "rnn_linattn_workspace_size",
           "rnn_linattn_fwd", "rnn_linattn_bwd", "rnn_linattn_step", "rms_norm",
           "rms_norm_backward", "quantize_weight", "input_proj_fp8", "linear_attention",
           "linear_attention_backward", "linear_attention_step"]

_native = None  # the compiled calls (csrc/binding.cpp), loaded with the library
_ENTRIES = ("rnn_rms_norm", "rnn_rms_norm_bwd_workspace_size", "rnn_rms_norm_bwd", "rnn_quantize_weight",
            "rnn_input_proj_fp8", "rnn_linattn_workspace_size", "rnn_linattn_fwd", "rnn_linattn_bwd",
            "rnn_linattn_step")


def _load():
    """The compiled calls, connected to the library that _lib.load() gives."""
    global _native
    lib = _lib.load()
    try:
        from . import _binding
    except ImportError as e:
        raise ImportError("the compiled calls of the language-model operators are missing or were built for "
                          "another PyTorch: build them with `python -m sequential_rnn_gb300.build`") from e
    _binding.connect(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _ENTRIES))
    _native = _binding
    return _binding


def _raise(status, where):
    from . import RnnError
    raise RnnError(status, where)


def _at(t):
    return t.data_ptr() if t is not None else None


def _handle(stream):
    """The raw handle of a stream; None: the current one."""
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _on(stream):
    """Makes `stream` the current one: what a call allocates then belongs to it, too."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream)


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
def rms_norm(x, weight, residual=None, *, eps=1e-6, quantize=False, train=False, stream=None):
    """h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight over the last dimension.

    x, residual [..., N] bf16 or fp32, weight [N] fp32.  Returns ``h`` (x itself
    without a residual), ``y`` (x's type; with ``quantize`` e4m3, NaN where y is not finite, and
    ``scale`` [..., ceil(N/128)] fp32) and with ``train`` the ``rstd`` [...] fp32 that
    ``rms_norm_backward`` takes.
    """
    if stream is not None:
        with _on(stream):
            return rms_norm(x, weight, residual, eps=eps, quantize=quantize, train=train)
    out = (_native or _load()).rms_norm(x, weight, residual, eps, quantize, train)
    if type(out) is int:
        _raise(out, "rnn_rms_norm")
    return out


def rms_norm_backward(dy, h, weight, rstd, *, dh=None, stream=None):
    """Gradient of ``rms_norm`` from its ``h`` and ``rstd``: ``dx`` (the gradient of x
    and of the residual, ``dh`` included) and ``dw`` [N] fp32."""
    if stream is not None:
        with _on(stream):
            return rms_norm_backward(dy, h, weight, rstd, dh=dh)
    out = (_native or _load()).rms_norm_backward(dy, h, weight, rstd, dh)
    if type(out) is int:
        _raise(out, "rnn_rms_norm_bwd")
    return out


# ------------------------------------------------------------ projection --
def quantize_weight(W, *, stream=None):
    """W [N, K] (bf16 or fp32) as e4m3 [N, K] and a scale for each 128 x 128 block."""
    if stream is not None:
        with _on(stream):
            return quantize_weight(W)
    out = (_native or _load()).quantize_weight(W)
    if type(out) is int:
        _raise(out, "rnn_quantize_weight")
    return out


def input_proj_fp8(xq, xs, Wq, Ws, bias=None, *, check=True, stream=None):
    """Wx = x W^T + bias from 8-bit operands through rnn_input_proj_fp8.

    xq [..., K], Wq [N, K] e4m3; xs [..., ceil(K/128)], Ws [ceil(N/128), ceil(K/128)]
    fp32 (``rms_norm(quantize=True)``'s and ``quantize_weight``'s); bias [N] fp32 or
    None -> [..., N] bf16, as ``input_proj`` gives it.
    """
    if stream is not None:
        with _on(stream):
            return input_proj_fp8(xq, xs, Wq, Ws, bias, check=check)
    out = (_native or _load()).input_proj_fp8(xq, xs, Wq, Ws, bias)
    if type(out) is int:
        _raise(out, "rnn_input_proj_fp8")
    if check:
        _read(out[1], "rnn_input_proj_fp8")
    return out[0]


# ------------------------------------------------------ linear attention --
def linear_attention(q, k, v, log_decay, *, state=None, lens=None, scale=None, check=True, stream=None):
    """S_t = exp(log_decay) S_{t-1} + k_t v_t^T, o_t = scale q_t S_t through rnn_linattn_fwd.

    q, k [T, B, NH, Dk], v [T, B, NH, Dv] bf16 or fp32 (strided views with a
    contiguous last dimension are taken as they are), log_decay [NH] fp32,
    state [B, NH, Dk, Dv] fp32 or None, lens [B] int32 or None (tokens of each row
    that count), scale Dk^-0.5 unless given.  Returns ``o`` [T, B, NH, Dv], ``state``
    (after the last token) and the ``workspace``.  A value that is not finite reaches its
    own and later tokens of its row and head and the state, never an output that does not
    depend on it.
    """
    if stream is not None:
        with _on(stream):
            return linear_attention(q, k, v, log_decay, state=state, lens=lens, scale=scale, check=check)
    out = (_native or _load()).linear_attention(q, k, v, log_decay, state, lens, scale)
    if type(out) is int:
        _raise(out, "rnn_linattn_fwd")
    if check:
        _read(out["workspace"], "rnn_linattn_fwd")
    return out


def linear_attention_backward(q, k, v, log_decay, do, *, state=None, dstate=None, lens=None,
                              scale=None, check=True, stream=None):
    """Gradients of ``linear_attention`` from its inputs, ``do`` [T, B, NH, Dv] (may be
    strided as they may) and ``dstate`` (of the final state, or None): ``dq``, ``dk``,
    ``dv`` and ``dstate`` (of the initial state)."""
    if stream is not None:
        with _on(stream):
            return linear_attention_backward(q, k, v, log_decay, do, state=state, dstate=dstate, lens=lens,
                                             scale=scale, check=check)
    out = (_native or _load()).linear_attention_backward(q, k, v, log_decay, do, state, dstate, lens, scale)
    if type(out) is int:
        _raise(out, "rnn_linattn_bwd")
    if check:
        _read(out["workspace"], "rnn_linattn_bwd")
    return out


def linear_attention_step(q, k, v, log_decay, state, *, slots=None, scale=None, stream=None):
    """One token for each row: q, k [B, NH, Dk], v [B, NH, Dv] against the cache ``state``
    [n_slots, NH, Dk, Dv] fp32, updated in place; row b uses state slots[b] (int32; None:
    state b).  A slot outside the cache gives zeros; no two rows may name the same one.
    Returns o [B, NH, Dv]."""
    if stream is not None:
        with _on(stream):
            return linear_attention_step(q, k, v, log_decay, state, slots=slots, scale=scale)
    out = (_native or _load()).linear_attention_step(q, k, v, log_decay, state, slots, scale)
    if type(out) is int:
        _raise(out, "rnn_linattn_step")
    return out
