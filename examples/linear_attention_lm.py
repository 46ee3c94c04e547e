"""A residual stack of linear-attention layers and one LSTM layer, served and trained with the
operators of ``sequential_rnn_gb300.lm``.

    python examples/linear_attention_lm.py          (needs a GB300)

Each layer reads the residual stream through the norm (which adds the previous layer's output to the
stream and writes 8 bits with scales in the same pass), projects it in 8 bits, and mixes over time:

    h, y8 = rms_norm(stream + out);  q, k, v = input_proj_fp8(y8);  o = linear_attention(q, k, v)
    out   = input_proj_fp8(rms_norm(o));      the LSTM layer takes the projection as its Wx instead

q, k and v are strided views of one projection.  A prompt runs all tokens at once; after it every
layer keeps a state ([NH, D, D] or the LSTM's h and c for each sequence), and a decoding step runs
the same layers on one token, captured once in a CUDA graph.
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


class Model:
    def __init__(self, NH=12, D=64, layers=("linear", "linear", "lstm"), seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.layers = [(LinearLayer if n == "linear" else LstmLayer)(NH, D, gen) for n in layers]
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


def main():
    NH, D, B, T, new = 12, 64, 16, 1024, 128
    m = Model(NH, D)
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


if __name__ == "__main__":
    main()
