"""A residual stack of linear-attention, gated and LSTM layers, served and trained with the
operators of ``sequential_rnn_gb300.lm``.

    python examples/linear_attention_lm.py          (needs a GB300)

Each layer reads the residual stream through the norm (which adds the previous layer's output to the
stream and writes 8 bits with scales in the same pass), projects it in 8 bits, and mixes over time:

    h, y8 = rms_norm(stream + out);  q, k, v = input_proj_fp8(y8);  o = linear_attention(q, k, v)
    out   = input_proj_fp8(rms_norm(o));      the LSTM layer takes the projection as its Wx instead,
                                              the gated layer (no recurrent matrix) as that of a scan

q, k and v are strided views of one projection; the rotary layer norms each head of q and k and turns it by its
token's position on their way to the attention.  A prompt runs all tokens at once; after it every
layer keeps a state ([NH, D, D], the rotary layer's with its sequences' positions, [NH, D], or the LSTM's h and c
for each sequence), and a decoding step runs the same layers on one token, captured once in a CUDA graph.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sequential_rnn_gb300 as S  # noqa: E402


def decays(NH, device="cuda"):
    """log(1 - 2^-1 .. 2^-9): heads that remember from two tokens to five hundred."""
    return torch.log1p(-torch.exp2(-torch.linspace(1, 9, NH, device=device)))


class LinearLayer:
    """Linear attention over NH heads of D, projections in 8 bits."""

    def __init__(self, NH, D, gen):
        d = NH * D
        self.NH, self.D = NH, D
        r = lambda *s: (torch.randn(s, generator=gen, device="cuda") * s[-1] ** -0.5).bfloat16()  # noqa: E731
        self.w_in, self.w_out = r(3 * d, d), r(d, d)
        self.in8, self.out8 = S.quantize_weight(self.w_in), S.quantize_weight(self.w_out)
        self.n_in, self.n_out = torch.ones(d, device="cuda"), torch.ones(d, device="cuda")
        self.decay = decays(NH)

    def _qkv(self, stream, out):
        n = S.rms_norm(stream, self.n_in, out, quantize=True)
        y = S.input_proj_fp8(n["y"], n["scale"], *self.in8, check=False)
        y = y.view(*y.shape[:-1], 3, self.NH, self.D)
        return n["h"], y.unbind(-3)

    def _out(self, o):
        n = S.rms_norm(o.flatten(-2), self.n_out, quantize=True)
        return S.input_proj_fp8(n["y"], n["scale"], *self.out8, check=False)

    def prompt(self, stream, out, lens=None):
        """stream, out [T, B, NH*D] -> (stream + out, this layer's output, its cache)."""
        stream, (q, k, v) = self._qkv(stream, out)
        a = S.linear_attention(q, k, v, self.decay, lens=lens, scale=self.D ** -0.5)
        return stream, self._out(a["o"]), a["state"]

    def step(self, stream, out, cache):
        """The same for one token [B, NH*D]; the cache is updated in place."""
        stream, (q, k, v) = self._qkv(stream, out)
        return stream, self._out(S.linear_attention_step(q, k, v, self.decay, cache, scale=self.D ** -0.5))


class RotaryLayer(LinearLayer):
    """Linear attention on queries and keys that are normed and turned by their positions."""

    def __init__(self, NH, D, gen):
        super().__init__(NH, D, gen)
        self.n_q, self.n_k = torch.ones(D, device="cuda"), torch.ones(D, device="cuda")
        self.freqs = S.rotary_frequencies(D)

    def _turned(self, q, k, at):
        return S.head_norm_rotary(q, k, self.n_q, self.n_k, self.freqs, at)

    def prompt(self, stream, out, lens=None):
        stream, (q, k, v) = self._qkv(stream, out)
        q, k = self._turned(q, k, None)
        a = S.linear_attention(q, k, v, self.decay, lens=lens, scale=self.D ** -0.5)
        T, B = q.shape[:2]
        at = torch.full((B,), T, dtype=torch.int32, device="cuda") if lens is None else lens.clamp(0, T)
        return stream, self._out(a["o"]), (a["state"], at)

    def step(self, stream, out, cache):
        state, at = cache
        stream, (q, k, v) = self._qkv(stream, out)
        q, k = self._turned(q, k, at)
        at += 1
        return stream, self._out(S.linear_attention_step(q, k, v, self.decay, state, scale=self.D ** -0.5))


class GatedLayer:
    """A gated linear recurrence on an 8-bit input projection: forget, input and output gates."""

    def __init__(self, NH, D, gen):
        d = NH * D
        self.NH, self.D = NH, D
        self.w = (torch.randn(3 * d, d, generator=gen, device="cuda") * d ** -0.5).bfloat16()
        self.w8 = S.quantize_weight(self.w)
        self.bias = torch.zeros(NH, 3, D, device="cuda")
        self.bias[:, 0] = torch.linspace(0, 6, D, device="cuda")  # memories from two tokens to four hundred
        self.n = torch.ones(d, device="cuda")

    def _wx(self, stream, out):
        n = S.rms_norm(stream, self.n, out, quantize=True)
        wx = S.input_proj_fp8(n["y"], n["scale"], *self.w8, self.bias.flatten(), check=False)
        return n["h"], wx.view(*wx.shape[:-1], self.NH, 3 * self.D)

    def prompt(self, stream, out, lens=None):
        stream, wx = self._wx(stream, out)
        f = S.gated_recurrence(wx, gates="fzo", lens=lens)
        return stream, f["y"].flatten(-2), f["state"]

    def step(self, stream, out, cache):
        stream, wx = self._wx(stream, out)
        return stream, S.gated_recurrence_step(wx, cache, gates="fzo").flatten(-2)


class LstmLayer:
    """The head-wise LSTM on an 8-bit input projection."""

    def __init__(self, NH, D, gen):
        d = NH * D
        self.NH, self.D = NH, D
        self.w = (torch.randn(4 * d, d, generator=gen, device="cuda") * d ** -0.5).bfloat16()
        self.w8 = S.quantize_weight(self.w)
        self.R = (torch.randn(NH, D, 4 * D, generator=gen, device="cuda") * D ** -0.5).bfloat16()
        self.n = torch.ones(d, device="cuda")

    def _run(self, stream, out, h0, c0):
        n = S.rms_norm(stream, self.n, out, quantize=True)
        wx = S.input_proj_fp8(n["y"], n["scale"], *self.w8, check=False)
        f = S.forward("lstm", wx.view(*wx.shape[:2], self.NH, -1), self.R, h0=h0, c0=c0, check=False)
        return n["h"], f["h_seq"].flatten(-2), (f["hT"], f["cT"])

    def prompt(self, stream, out, lens=None):
        if lens is not None:
            raise ValueError("the LSTM layer takes sequences of one length")
        return self._run(stream, out, None, None)

    def step(self, stream, out, cache):
        s, o, new = self._run(stream[None], None if out is None else out[None], *cache)
        for old, x in zip(cache, new):
            old.copy_(x)
        return s[0], o[0]


LAYERS = {"linear": LinearLayer, "rotary": RotaryLayer, "gated": GatedLayer, "lstm": LstmLayer}


class Model:
    def __init__(self, NH=12, D=64, layers=("linear", "linear", "lstm"), seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.layers = [LAYERS[n](NH, D, gen) for n in layers]
        self.norm = torch.ones(NH * D, device="cuda")

    def prompt(self, x, lens=None):
        """x [T, B, NH*D] bf16 -> (normed stream [T, B, NH*D], the layers' caches)."""
        out, caches = None, []
        for layer in self.layers:
            x, out, c = layer.prompt(x, out, lens)
            caches.append(c)
        return S.rms_norm(x, self.norm, out)["y"], caches

    def step(self, x, caches):
        """One token x [B, NH*D]; the caches are updated in place."""
        out = None
        for layer, c in zip(self.layers, caches):
            x, out = layer.step(x, out, c)
        return S.rms_norm(x, self.norm, out)["y"]

    def graph(self, caches, B):
        """A decoding step on fixed buffers as a CUDA graph: (x, y, replay).  The caches are restored after
        the warm-up."""
        x = torch.zeros((B, self.norm.numel()), dtype=torch.bfloat16, device="cuda")
        flat = [t for c in caches for t in (c if isinstance(c, tuple) else (c,))]
        keep = [t.clone() for t in flat]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.step(x, caches)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = self.step(x, caches)
        for t, k in zip(flat, keep):
            t.copy_(k)
        return x, y, g.replay


def mixer_loss(x, w, decay, NH, D, target):
    """Loss sum(o target) of norm -> linear attention with q, k, v taken from the norm's output [T, B, 3*NH*D],
    and its gradients (dx, dw)."""
    n = S.rms_norm(x, w, train=True)
    q, k, v = n["y"].view(*x.shape[:2], 3, NH, D).unbind(2)
    a = S.linear_attention(q, k, v, decay)
    loss = (a["o"].float() * target.float()).sum()
    g = S.linear_attention_backward(q, k, v, decay, target)
    dy = torch.stack([g["dq"], g["dk"], g["dv"]], 2).flatten(2)
    d = S.rms_norm_backward(dy, n["h"], w, n["rstd"])
    return loss, d["dx"], d["dw"]


def training_step(x, w, w_q, w_k, freqs, decay, NH, D, target, limit):
    """Two mixers side by side on one norm of x [T, B, 5*NH*D]: its first three parts are the queries, keys and values of
    rotated linear attention, the others the gates of a recurrence; loss sum((o + y) target).  Returns the loss,
    the weights' gradients clipped to a common norm of `limit`, dx, and that norm before."""
    T, B, d = *x.shape[:2], NH * D
    n = S.rms_norm(x, w, train=True)
    q, k, v = n["y"][..., :3 * d].view(T, B, 3, NH, D).unbind(2)
    wx = n["y"][..., 3 * d:].contiguous().view(T, B, NH, 2 * D)
    qt, kt = S.head_norm_rotary(q, k, w_q, w_k, freqs)
    a = S.linear_attention(qt, kt, v, decay)
    f = S.gated_recurrence(wx, train=True)
    loss = ((a["o"].float() + f["y"].float()) * target.float()).sum()
    ga = S.linear_attention_backward(qt, kt, v, decay, target)
    gf = S.gated_recurrence_backward(wx, f["stash"], target)
    gr = S.head_norm_rotary_backward(q, k, w_q, w_k, freqs, None, ga["dq"], ga["dk"])
    dy = torch.cat([gr["dq"].flatten(2), gr["dk"].flatten(2), ga["dv"].flatten(2), gf["dWx"].flatten(2)], -1)
    dn = S.rms_norm_backward(dy, n["h"], w, n["rstd"])
    grads = {"dw": dn["dw"], "dw_q": gr["dwq"], "dw_k": gr["dwk"]}
    norm = S.clip_grad_norm(list(grads.values()), limit)
    return loss, grads, dn["dx"], norm


def main():
    NH, D, B, T, new = 12, 64, 16, 1024, 128
    m = Model(NH, D, layers=("rotary", "gated", "lstm"))
    x = torch.randn(T, B, NH * D, device="cuda").bfloat16()
    for _ in range(3):
        m.prompt(x)
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(4)]
    ev[0].record()
    y, caches = m.prompt(x)
    ev[1].record()
    xin, yout, replay = m.graph(caches, B)
    tok = y[-1]
    ev[2].record()
    for _ in range(new):
        xin.copy_(tok)
        replay()
        tok = yout
    ev[3].record()
    torch.cuda.synchronize()
    ms = ev[0].elapsed_time(ev[1])
    us = ev[2].elapsed_time(ev[3]) * 1e3 / new
    print(f"prompt: {T} tokens x {B} sequences in {ms:.2f} ms ({T * B / ms / 1e3:.1f} M tokens/s); "
          f"decoding: {us:.0f} us a step of {B} tokens")
    for _ in range(2):
        loss, dx, dw = mixer_loss(torch.randn(T, B, 3 * NH * D, device="cuda").bfloat16(),
                                  torch.ones(3 * NH * D, device="cuda"), decays(NH), NH, D,
                                  torch.randn(T, B, NH, D, device="cuda").bfloat16())
    print(f"training: loss {loss.item():.4g}, |dx| {dx.float().norm().item():.4g}, |dw| {dw.norm().item():.4g}")
    one = torch.ones(D, device="cuda")
    loss, grads, _, norm = training_step(torch.randn(T, B, 5 * NH * D, device="cuda").bfloat16(),
                                         torch.ones(5 * NH * D, device="cuda"), one, one, S.rotary_frequencies(D),
                                         decays(NH), NH, D, torch.randn(T, B, NH, D, device="cuda").bfloat16(), 1.0)
    print(f"both mixers: loss {loss.item():.4g}, weights' gradients of norm {norm.item():.4g} clipped to "
          f"{S.grad_norm(list(grads.values())).item():.4g}")


if __name__ == "__main__":
    main()
