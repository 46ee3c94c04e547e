"""What is measured of the operators around a recurrent language model's mixers and
its training: the gated linear recurrence over time (prompts, training, single
tokens), the norm of each query's and key's head with the rotation by its position
(and its gradient), and the clipping of all gradients by their common norm.

``own`` false: the plain forms, elementary torch operations in fp32 (angles and the
gradients' common sum in fp64).  ``own`` true: the framework's calls.  Head shapes and
widths are those of the framework's workloads (12 heads of 64, 6 of 128, 4 of 256).
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
BASE = 10000.0
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases --
def _gated(op, t, b, nh, d, gates, ragged=False, dtype="bf16"):
    return {"op": op, "t": t, "b": b, "nh": nh, "d": d, "gates": gates, "ragged": ragged, "dtype": dtype}


def _rotary(op, t, b, nq, nk, d, rot, interleaved=False, dtype="bf16"):
    return {"op": op, "t": t, "b": b, "nq": nq, "nk": nk, "d": d, "rot": rot, "interleaved": interleaved,
            "dtype": dtype}


def _clip(layers, nh, d, g, extra=0, dtype="bf16"):
    return {"op": "clip", "layers": layers, "nh": nh, "d": d, "g": g, "extra": extra, "dtype": dtype}


def listed():
    return [
        # one token for each of 16 sequences out of a cache of 20 states, 12 x 64 heads
        dict(_gated("gated_step", 1, 16, 12, 64, "fz"), name="gated_token"),
        # one token for each of 160 sequences, all four gates, 4 x 256 heads
        dict(_gated("gated_step", 1, 160, 4, 256, "ifzo"), name="gated_tokens"),
        # a few short prompts of different lengths
        dict(_gated("gated", 333, 5, 12, 64, "ifzo", ragged=True), name="gated_ragged"),
        # one long prompt
        dict(_gated("gated", 16384, 1, 12, 64, "fz"), name="gated_long"),
        # training, forward and backward: T 1024 x B 16 on 12 x 64 heads
        dict(_gated("gated_train", 1024, 16, 12, 64, "fzo"), name="gated_train"),
        # the same in fp32 on 6 x 128 heads with an odd length
        dict(_gated("gated_train", 2001, 4, 6, 128, "ifzo", dtype="f32"), name="gated_train_f32"),
        # queries and keys of one token for each of 16 sequences
        dict(_rotary("rotary", 1, 16, 12, 12, 64, 64), name="rotary_token"),
        # of a batch of prompts, T 1024 x B 16
        dict(_rotary("rotary", 1024, 16, 12, 12, 64, 64), name="rotary_prompt"),
        # gradient for a short batch of wide heads that share keys, half of each head rotated
        dict(_rotary("rotary_grad", 101, 3, 4, 2, 256, 128, interleaved=True), name="rotary_grad_ragged"),
        # gradient in training on 6 x 128 heads with an odd length
        dict(_rotary("rotary_grad", 2001, 4, 6, 6, 128, 128), name="rotary_grad"),
        # the gradients of one GRU layer of 6 x 128
        dict(_clip(1, 6, 128, 3), name="clip_layer"),
        # of 12 sLSTM layers of 4 x 256 with an embedding
        dict(_clip(12, 4, 256, 4, extra=32003), name="clip_stack"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = [(12, 64), (6, 128), (4, 256), (3, 32), (1, 768), (5, 40), (2, 33)]


def draw(rng):
    op = rng.choice(["gated_step", "gated", "gated", "gated_train", "gated_train", "rotary", "rotary", "rotary_grad",
                     "rotary_grad", "clip"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "clip":
        nh, d = rng.choice(HEADS)
        return _clip(_log(rng, 1, 12), nh, d, rng.choice([3, 4]), rng.choice([0, _log(rng, 1, 32003)]), dtype)
    if op.startswith("gated"):
        nh, d = rng.choice(HEADS)
        gates = rng.choice(["fz", "fzo", "ifzo"])
        if op == "gated_step":
            return _gated(op, 1, _log(rng, 1, 160), nh, d, gates, dtype=dtype)
        most = 16384 * 768 // (nh * d) // (2 if op == "gated_train" and dtype == "f32" else 1)
        t = _log(rng, 1, min(16384, most))
        b = _log(rng, 1, max(1, min(32, most // t)))
        return _gated(op, t, b, nh, d, gates, rng.random() < 0.5, dtype)
    nq, d = rng.choice([(12, 64), (6, 128), (4, 256), (3, 32), (5, 40), (7, 96), (2, 34)])
    nk = rng.choice([nq, nq, 1, 2])
    rot = rng.choice([d, d, d // 4 * 2, 2])
    most = 16384 * 768 // (nq * d)
    t = rng.choice([1, _log(rng, 1, min(16384, most))])
    b = _log(rng, 1, max(1, min(160, most // t)))
    return _rotary(op, t, b, nq, nk, d, rot, rng.random() < 0.3, dtype)


def _shapes(case):
    """Gradients of `layers` layers (input weight, recurrent weight, bias, norm), an embedding and a scalar."""
    nh, d, g = case["nh"], case["d"], case["g"]
    n, low = nh * d, DTYPES[case["dtype"]]
    out = []
    for _ in range(case["layers"]):
        out += [((g * n, n), low), ((nh, d, g * d), torch.float32), ((nh, g * d), torch.float32),
                ((n,), torch.float32)]
    if case["extra"]:
        out += [((case["extra"], n), low), ((1,), torch.float32)]
    return out


def work(case):
    op = case["op"]
    if op == "clip":  # every gradient in and out
        sizes = [(math.prod(s), 4 if dt == torch.float32 else 2) for s, dt in _shapes(case)]
        return {"bytes": 2 * sum(n * e for n, e in sizes), "flops": 3.0 * sum(n for n, _ in sizes)}
    e = 4 if case["dtype"] == "f32" else 2
    if op.startswith("rotary"):
        t, b, heads, d = case["t"], case["b"], case["nq"] + case["nk"], case["d"]
        n = t * b * heads * d
        fixed = 8 * d + 4 * case["rot"] + 4 * b
        if op == "rotary":  # q, k in and out
            return {"bytes": 2 * n * e + fixed, "flops": 6.0 * n}
        return {"bytes": 3 * n * e + fixed + 8 * d, "flops": 14.0 * n}
    t, b, n, g = case["t"], case["b"], case["nh"] * case["d"], len(case["gates"])
    if op == "gated_step":
        return {"bytes": b * n * ((g + 1) * e + 8), "flops": 10.0 * b * n}
    tokens = sum(_lens(case)) if case["ragged"] else t * b
    if op == "gated":  # the gates in, y out, both states
        return {"bytes": tokens * n * g * e + t * b * n * e + 8 * b * n, "flops": 10.0 * tokens * n}
    # the gates and dy in, y and the gates' gradients out, the states and their gradients
    return {"bytes": tokens * n * (g + 1) * e + t * b * n * (g + 1) * e + 16 * b * n, "flops": 30.0 * tokens * n}


# ----------------------------------------------------------------- inputs --
def _lens(case):
    """Tokens of each row that count: from the whole length down to none."""
    t, b = case["t"], case["b"]
    return [t - (t * i) // max(1, b - 1) for i in range(b)] if b > 1 else [t - t // 3]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)

    op, st = case["op"], {"op": case["op"], "case": case}
    if op == "clip":
        st["grads"] = [normal(*s, dtype=dt) for s, dt in _shapes(case)]
        # a common norm about three times the limit, spread over the tensors unevenly
        total = math.sqrt(sum(math.prod(s) for s, _ in _shapes(case)))
        for i, x in enumerate(st["grads"]):
            x *= (1 + i % 5) / total
        st["limit"] = 1.0
        return st
    dtype = DTYPES[case["dtype"]]
    if op.startswith("rotary"):
        t, b, nq, nk, d = (case[k] for k in ("t", "b", "nq", "nk", "d"))
        # q, k and v as one projection writes them, side by side for each token
        qkv = normal(t, b, (nq + 2 * nk) * d, dtype=dtype, scale=2.0)
        st["q"] = qkv[..., :nq * d].view(t, b, nq, d)
        st["k"] = qkv[..., nq * d:(nq + nk) * d].view(t, b, nk, d)
        st["wq"], st["wk"] = 1.0 + normal(d, scale=0.1), 1.0 + normal(d, scale=0.1)
        j = torch.arange(case["rot"] // 2, dtype=torch.float64, device=DEV)
        st["freqs"] = torch.exp(j * (-2.0 / case["rot"] * math.log(BASE)))
        # where each row's first token stands: long conversations among short ones
        far = torch.exp(torch.rand(b, generator=g, device=DEV) * math.log(1e6))
        st["start"] = far.int() - 1
        if op == "rotary_grad":
            st["dq"] = normal(t, b, nq, d, dtype=dtype, scale=0.01)
            st["dk"] = normal(t, b, nk, d, dtype=dtype, scale=0.01)
        return st
    t, b, nh, d, names = (case[k] for k in ("t", "b", "nh", "d", "gates"))
    # forget gates from a memory of a few tokens to some hundred, as a trained layer's channels spread
    wx = normal(t, b, nh, len(names), d)
    wx[..., names.index("f"), :] += torch.linspace(0.0, 5.0, nh * d, device=DEV).view(nh, d)
    wx = wx.to(dtype).view(t, b, nh, len(names) * d)
    if op == "gated_step":
        slots = b + -(-b // 4)
        st["Wx"] = wx[0]
        st["cache"] = normal(slots, nh, d)
        st["slots"] = torch.randperm(slots, generator=g, device=DEV)[:b].int()
        st["at"] = st["slots"].long()
        return st
    st["Wx"], st["s0"] = wx, normal(b, nh, d)
    st["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device=DEV) if case["ragged"] else None
    if op == "gated_train":
        st["dy"] = normal(t, b, nh, d, dtype=dtype, scale=0.1)
        st["ds"] = normal(b, nh, d, scale=0.1)
    return st


# ------------------------------------------------------------ plain forms --
def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _split(wx, names):
    """{gate: [..., NH, D] in fp32} of [..., NH, G*D]."""
    parts = wx.float().unflatten(-1, (len(names), -1)).unbind(-2)
    return dict(zip(names, parts))


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the first dimension, h_{-1} = 0, by doubling."""
    n = 1
    while n < a.shape[0]:
        b = torch.cat([b[:n], b[n:] + a[n:] * b[:-n]])
        a = torch.cat([a[:n], a[n:] * a[:-n]])
        n *= 2
    return b


def _live(st):
    t = st["Wx"].shape[0]
    if st["lens"] is None:
        return torch.ones((t, 1, 1, 1), dtype=torch.bool, device=DEV)
    return (torch.arange(t, device=DEV)[:, None] < st["lens"][None])[..., None, None]


def _plain_gated(st):
    """Everything that the backward pass uses, too."""
    p = _split(st["Wx"], st["case"]["gates"])
    live, zero = _live(st), torch.zeros((), device=DEV)
    keep, take = _sigmoid(p["f"]), _sigmoid(-p["f"])
    gain = _sigmoid(p["i"]) if "i" in p else take
    a = torch.where(live, keep, torch.ones((), device=DEV))
    u = torch.where(live, gain * p["z"], zero)
    u[0] += a[0] * st["s0"]
    h = _scan(a, u)
    o = _sigmoid(p["o"]) if "o" in p else None
    y = torch.where(live, h if o is None else o * h, zero)
    return p, live, keep, take, gain, a, h, o, y


def _plain_prompt(st):
    h, y = [_plain_gated(st)[i] for i in (6, 8)]
    return {"y": y.to(st["Wx"].dtype), "state": h[-1].clone()}


def _plain_train(st):
    p, live, keep, take, gain, a, h, o, y = _plain_gated(st)
    zero = torch.zeros((), device=DEV)
    dy = torch.where(live, st["dy"].float(), zero)
    e = dy.clone() if o is None else dy * o
    e[-1] += st["ds"]
    up = torch.cat([torch.ones_like(a[:1]), a[1:].flip(0)])  # what dh_{t+1} is weighted with, in reversed time
    dh = _scan(up, e.flip(0)).flip(0)
    before = torch.cat([st["s0"][None], h[:-1]])
    g = {"z": dh * gain}
    if "i" in p:
        g["f"] = dh * before * keep * take
        g["i"] = dh * p["z"] * gain * _sigmoid(-p["i"])
    else:
        g["f"] = dh * (before - p["z"]) * keep * take
    if o is not None:
        g["o"] = dy * h * o * _sigmoid(-p["o"])
    dwx = torch.stack([torch.where(live, g[n], zero) for n in st["case"]["gates"]], -2).flatten(-2)
    dt = st["Wx"].dtype
    return {"y": y.to(dt), "state": h[-1].clone(), "dWx": dwx.to(dt), "dstate": a[0] * dh[0]}


def _plain_step(st):
    p = _split(st["Wx"], st["case"]["gates"])
    take = _sigmoid(-p["f"])
    gain = _sigmoid(p["i"]) if "i" in p else take
    h = _sigmoid(p["f"]) * st["cache"][st["at"]] + gain * p["z"]
    st["cache"][st["at"]] = h
    y = _sigmoid(p["o"]) * h if "o" in p else h
    return {"y": y.to(st["Wx"].dtype), "cache": st["cache"]}


def _angles(st, dtype):
    """cos and sin [T, B, 1, rot / 2], the angles in fp64."""
    t = st["q"].shape[0]
    at = st["start"].double()[None] + torch.arange(t, dtype=torch.float64, device=DEV)[:, None]
    x = (at[..., None] * st["freqs"])[:, :, None]
    return torch.cos(x).to(dtype), torch.sin(x).to(dtype)


def _turn(x, cos, sin, interleaved):
    """Pairs of the first columns rotated, the others as they are."""
    n = 2 * cos.shape[-1]
    r, rest = x[..., :n], x[..., n:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        out = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., :n // 2], r[..., n // 2:]
        out = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([out, rest], -1)


def _plain_rotary(st):
    cos, sin = _angles(st, torch.float32)
    out = {}
    for n in "qk":
        x = st[n].float()
        y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * st["w" + n]
        out[n] = _turn(y, cos, sin, st["case"]["interleaved"]).to(st[n].dtype)
    return out


def _plain_rotary_grad(st):
    cos, sin = _angles(st, torch.float32)
    out = {}
    for n in "qk":
        x = st[n].float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        dy = _turn(st["d" + n].float(), cos, -sin, st["case"]["interleaved"])
        xh, wdy = x * r, dy * st["w" + n]
        out["d" + n] = (r * (wdy - xh * (wdy * xh).mean(-1, keepdim=True))).to(st[n].dtype)
        out["dw" + n] = (dy * xh).sum((0, 1, 2))
    return out


def _tighter(st):
    """The limit of this pass; a later pass, on gradients that this one has clipped, clips as well."""
    now = st["limit"]
    st["limit"] = now * 0.999
    return now


def _clipped(norm, grads):
    return {"norm": norm, **{str(i): x for i, x in enumerate(grads)}}


def _plain_clip(st):
    limit = _tighter(st)
    total = torch.zeros((), dtype=torch.float64, device=DEV)
    for x in st["grads"]:
        total = total + x.float().square().sum(dtype=torch.float64)
    norm = total.sqrt()
    by = torch.where(norm > limit, limit / norm, torch.ones_like(norm)).float()
    for x in st["grads"]:
        x.copy_(x.float() * by)
    return _clipped(norm.float(), st["grads"])


def _plain(st):
    return {"gated": _plain_prompt, "gated_train": _plain_train, "gated_step": _plain_step, "rotary": _plain_rotary,
            "rotary_grad": _plain_rotary_grad, "clip": _plain_clip}[st["op"]](st)


# --------------------------------------------------------- the framework's --
def _framework(st):
    import sequential_rnn_gb300 as S
    op, case = st["op"], st["case"]
    if op == "clip":
        return _clipped(S.clip_grad_norm(st["grads"], _tighter(st)), st["grads"])
    if op == "rotary":
        q, k = S.head_norm_rotary(st["q"], st["k"], st["wq"], st["wk"], st["freqs"], st["start"], eps=EPS,
                                  interleaved=case["interleaved"])
        return {"q": q, "k": k}
    if op == "rotary_grad":
        return S.head_norm_rotary_backward(st["q"], st["k"], st["wq"], st["wk"], st["freqs"], st["start"], st["dq"],
                                           st["dk"], eps=EPS, interleaved=case["interleaved"])
    if op == "gated_step":
        y = S.gated_recurrence_step(st["Wx"], st["cache"], gates=case["gates"], slots=st["slots"])
        return {"y": y, "cache": st["cache"]}
    train = op == "gated_train"
    out = S.gated_recurrence(st["Wx"], gates=case["gates"], state=st["s0"], lens=st["lens"], train=train,
                             check=False)
    res = {"y": out["y"], "state": out["state"]}
    if train:
        g = S.gated_recurrence_backward(st["Wx"], out["stash"], st["dy"], gates=case["gates"], dstate=st["ds"],
                                        lens=st["lens"], check=False)
        res.update(dWx=g["dWx"], dstate=g["dstate"])
    return res


def run(state):
    return _framework(state) if own else _plain(state)


# ---------------------------------------------------------- in 64 bits --
def _exact_gated(st):
    """Token by token, as the recurrence defines it."""
    names, dt = st["case"]["gates"], torch.float64
    wx = st["Wx"].to(dt).unflatten(-1, (len(names), -1))
    p = {n: wx[..., i, :] for i, n in enumerate(names)}
    f = torch.special.expit(p["f"])
    gain = torch.special.expit(p["i"] if "i" in p else -p["f"])
    o = torch.special.expit(p["o"]) if "o" in p else None
    if st["op"] == "gated_step":
        cache = st["cache"].to(dt)
        h = f * cache[st["at"]] + gain * p["z"]
        cache[st["at"]] = h
        return {"y": h if o is None else o * h, "cache": cache}
    t, b = wx.shape[:2]
    lens = [t] * b if st["lens"] is None else st["lens"].tolist()
    on = [torch.tensor([n > i for n in lens], device=DEV)[:, None, None] if min(lens) <= i else None
          for i in range(t)]
    h, hs, ys = st["s0"].to(dt), [], []
    for i in range(t):
        hs.append(h)
        new = f[i] * h + gain[i] * p["z"][i]
        y = new if o is None else o[i] * new
        h = new if on[i] is None else torch.where(on[i], new, h)
        ys.append(y if on[i] is None else y * on[i])
    out = {"y": torch.stack(ys), "state": h}
    if st["op"] == "gated":
        return out
    dh, dwx = st["ds"].to(dt), torch.zeros_like(wx)
    dy = st["dy"].to(dt)
    at = {n: i for i, n in enumerate(names)}
    for i in reversed(range(t)):
        d = dh + (dy[i] if o is None else dy[i] * o[i])
        g = {"z": d * gain[i]}
        slope = f[i] * torch.special.expit(-p["f"][i])
        if "i" in p:
            g["f"] = d * hs[i] * slope
            g["i"] = d * p["z"][i] * gain[i] * torch.special.expit(-p["i"][i])
        else:
            g["f"] = d * (hs[i] - p["z"][i]) * slope
        if o is not None:
            g["o"] = dy[i] * (f[i] * hs[i] + gain[i] * p["z"][i]) * o[i] * torch.special.expit(-p["o"][i])
        for n, x in g.items():
            dwx[i, :, :, at[n]] = x if on[i] is None else x * on[i]
        dh = f[i] * d if on[i] is None else torch.where(on[i], f[i] * d, dh)
    out.update(dWx=dwx.flatten(-2), dstate=dh)
    return out


def _exact_rotary(st):
    case, out = st["case"], {}
    t, half = st["q"].shape[0], case["rot"] // 2
    at = st["start"].long()[None] + torch.arange(t, device=DEV)[:, None]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                       at.double()[..., None] * st["freqs"])[:, :, None]  # e^(i angle)
    cols = torch.arange(2 * half, device=DEV)
    one, two = (cols[0::2], cols[1::2]) if case["interleaved"] else (cols[:half], cols[half:])

    def rotated(x, by):
        c = torch.complex(x[..., one], x[..., two]) * by
        x = x.clone()
        x[..., one], x[..., two] = c.real, c.imag
        return x

    for n in "qk":
        x, w = st[n].double(), st["w" + n].double()
        r = (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).pow(-0.5)
        if case["op"] == "rotary":
            out[n] = rotated(x * r * w, turn)
            continue
        dy = rotated(st["d" + n].double(), turn.conj())
        along = (dy * w * x).sum(-1, keepdim=True) * r.pow(3) / x.shape[-1]
        out["d" + n] = dy * w * r - x * along
        out["dw" + n] = torch.einsum("tbhd,tbhd,tbh->d", dy, x, r[..., 0])
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "clip":
        norm = math.sqrt(math.fsum(x.double().pow(2).sum().item() for x in st["grads"]))
        by = st["limit"] / norm if norm > st["limit"] else 1.0
        return _clipped(torch.tensor(norm, dtype=torch.float64, device=DEV), [x.double() * by for x in st["grads"]])
    return _exact_rotary(st) if case["op"].startswith("rotary") else _exact_gated(st)
