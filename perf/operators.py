"""Cases and plain forms of the residual-stream operators: RMSNorm with the
residual's addition (and its gradient), the same with an 8-bit output and
scales, 8-bit activation checkpoints, and the norm's forward and backward
that write and read such a checkpoint.

With x, res [M, N] of one type, w [N], f32 arithmetic, rx the rounding to x's
type, r8 the rounding to 8 bits, w' = w (or 1 + w, expression 2):

  s = rx(x + res)                    the residual stream, held in x's type
  r = 1 / sqrt(mean_j s^2 + eps)     one f32 a row
  y = rx(w' s r)                     expression 0: rx(w rx(s r))
  8-bit output, over each group of columns (or the row, group 0):
      scale = max(max|w' s r| / qmax, 2^-100),  q = r8(w' s r / scale)
  checkpoint of s, over each group:
      scale = max(max|s| (1 / qmax), 2^-100),   q = r8(s (1 / scale))
  backward, dy and ds the gradients of y and s, xh = s r (or q scale r):
      dn = dy w'  (expression 0: rx(dy w), and rx(dy rx(xh)) in dw; not from a checkpoint)
      dx = rx(ds + r (dn - xh mean_j(dn xh)))   of x and of res alike
      dw = sum_i dy xh
"""
import math

import torch

own = False

EPS = 1e-6
FLOOR = 2.0 ** -100
QMAX = {"e4m3": 448.0, "int8": 127.0}
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
Q_TYPES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}

_library = None


def _gbn():
    global _library
    if _library is None:
        import normalization_layers_fwd_gb300 as _library
    return _library


# ------------------------------------------------------------------- cases

def _case(name, op, M, N, type, wtype, variant, group=0, q="e4m3", pad=0):
    c = {"op": op, "M": M, "N": N, "type": type, "wtype": wtype, "variant": variant}
    if op not in ("add", "bwd"):
        c.update(group=group, q=q)
    if pad:
        c["pad"] = pad
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token in generation: the launch counts, not the 32 KB
        _case("add, one token", "add", 1, 4096, "bf16", "bf16", 0),
        # a training step's forward at the widest model of the sweep; x is a slice of a wider projection
        _case("add, training step", "add", 16384, 8192, "bf16", "f32", 1, pad=64),
        # a batch of 64 sequences, one token each, into an 8-bit product with one scale a token
        _case("8-bit out, decode batch", "quant", 64, 8192, "bf16", "bf16", 1),
        # a prompt's prefill into an 8-bit product with a scale per 128 columns
        _case("8-bit out, prefill", "quant", 16384, 4096, "bf16", "bf16", 2, 128),
        # a packed batch of ragged length at an odd width
        _case("backward, ragged odd width", "bwd", 4097, 1001, "f16", "f16", 2),
        # the gradient at the RMSNorm training shape, doubled in width
        _case("backward, training step", "bwd", 16384, 4096, "bf16", "bf16", 0),
        # a small f32 layer's input kept in 8 bits and read back
        _case("pack and unpack, small f32", "pack", 512, 2048, "f32", "f32", 1, 32),
        # an input kept for the backward of another layer
        _case("pack and unpack, training", "pack", 32768, 4096, "bf16", "bf16", 1, 128),
        # a short micro-batch in half precision, one scale a row
        _case("checkpoint forward, short", "ckpt_fwd", 384, 1024, "f16", "f32", 1, 0),
        # the training forward that also leaves the checkpoint
        _case("checkpoint forward, training", "ckpt_fwd", 16384, 4096, "bf16", "bf16", 0, 128),
        # a ragged micro-batch, rows that are not whole vectors
        _case("checkpoint backward, ragged", "ckpt_bwd", 3001, 2050, "bf16", "bf16", 1, 64),
        # the training backward from an int8 checkpoint
        _case("checkpoint backward, training", "ckpt_bwd", 16384, 8192, "bf16", "bf16", 1, 128, "int8"),
    ]


def draw(rng):
    """One more case: rows from 1 to 65536 and widths from 32 to 16384 (f32 to
    8192), spread over their logarithms, a third of the widths odd."""
    op = rng.choice(("add", "quant", "bwd", "pack", "ckpt_fwd", "ckpt_bwd"))
    type = rng.choice(("bf16", "bf16", "bf16", "f16", "f32"))
    N = int(round(2 ** rng.uniform(5, 13 if type == "f32" else 14)))
    shape = rng.randrange(3)
    N = N | 1 if shape == 0 else max(32, N // 8 * 8) if shape == 1 else N
    N = min(N, 8192 if type == "f32" else 16384)
    # the work of a pass stays below the largest listed one's
    room = 2 ** 25 if type == "f32" else 2 ** 26
    M = int(round(2 ** rng.uniform(0, min(16.0, math.log2(room / N)))))
    variant = rng.randrange(3)
    wtype = type if variant == 0 else rng.choice((type, "f32"))
    q = rng.choice(("e4m3", "int8")) if op == "ckpt_bwd" else "e4m3"
    pad = 16 if op in ("add", "quant", "ckpt_fwd") and N % 8 == 0 and rng.random() < 0.25 else 0
    return _case(None, op, M, N, type, wtype, variant, rng.choice((0, 32, 64, 128)), q, pad)


def _ngroups(case):
    g = case["group"]
    return 1 if g == 0 else -(-case["N"] // g)


def work(case):
    M, N, e = case["M"], case["N"], BYTES[case["type"]]
    E, op = M * N, case["op"]
    wb = N * BYTES[case["wtype"]]
    scales = 4 * M * _ngroups(case) if "group" in case else 0
    if op == "add":
        return {"bytes": 4 * E * e + wb + 4 * M, "flops": 6 * E}
    if op == "quant":
        return {"bytes": E * (3 * e + 1) + wb + scales, "flops": 7 * E}
    if op == "bwd":
        return {"bytes": 4 * E * e + 2 * wb + 4 * M, "flops": 11 * E}
    if op == "pack":
        return {"bytes": 2 * (E * (e + 1) + scales), "flops": 3 * E}
    if op == "ckpt_fwd":
        return {"bytes": E * (4 * e + 1) + wb + scales + 4 * M, "flops": 8 * E}
    return {"bytes": E * (3 * e + 1) + 2 * wb + scales + 4 * M, "flops": 12 * E}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    M, N, t = case["M"], case["N"], TYPES[case["type"]]
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, mean=0.0, std=1.0):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(std).add_(mean)

    st = dict(case)
    w = normal(N, mean=0.0, std=0.1) if case["variant"] == 2 else normal(N, mean=1.0, std=0.1)
    st["w"] = w.to(TYPES[case["wtype"]])
    # a residual stream: a few columns run several times larger than the rest
    gain = torch.where(torch.rand(N, generator=gen, device="cuda") < 0.01, 8.0, 1.0)
    stream = normal(M, N, std=1.5).mul_(gain).to(t)
    op = case["op"]
    if op in ("add", "quant", "ckpt_fwd"):
        st["res"] = stream
        x = normal(M, N + case.get("pad", 0)).to(t)
        st["x"] = x[:, :N] if case.get("pad") else x
        return st
    if op == "pack":
        st["x"] = stream
        return st
    st["dy"] = normal(M, N, std=0.02).to(t)
    st["ds"] = normal(M, N, std=0.02).to(t)
    st["rstd"] = torch.rsqrt(stream.float().square().mean(-1) + EPS)
    if op == "bwd":
        st["s"] = stream
    else:
        st["c"], st["cscale"] = _pack(stream, case["q"], case["group"])
    return st


# -------------------------------------------------------------- plain form

def _groups(v, group):
    """v [M, N] as [M, groups, columns of a group], the last one filled up with zeros."""
    M, N = v.shape
    g = group or N
    n = -(-N // g)
    if n * g != N:
        v = torch.nn.functional.pad(v, (0, n * g - N))
    return v.view(M, n, g)


def _spread(scale, N, group):
    """scale [M, groups] at each of the N columns."""
    return scale if group == 0 else scale.repeat_interleave(group, dim=1)[:, :N]


def _round8(v, q):
    return v.to(torch.float8_e4m3fn) if q == "e4m3" else v.round().to(torch.int8)


def _pack(x, q, group):
    x = x.float()
    amax = _groups(x.abs(), group).amax(-1)
    scale = torch.clamp(amax * (1.0 / QMAX[q]), min=FLOOR)
    return _round8(x * _spread(1.0 / scale, x.shape[1], group), q), scale


def _weight(st):
    w = st["w"].float()
    return 1.0 + w if st["variant"] == 2 else w


def _stream(st):
    s = (st["x"].float() + st["res"].float()).to(TYPES[st["type"]])
    f = s.float()
    return s, f, torch.rsqrt(f.square().mean(-1) + EPS)


def _norm(st, f, r):
    t = TYPES[st["type"]]
    n = f * r[:, None]
    if st["variant"] == 0:
        n = n.to(t).float()
    return (n * _weight(st)).to(t)


def _gradients(st, xh, rounded):
    """dx and dw from xh; rounded: expression 0's rounding points."""
    t, dy, r = TYPES[st["type"]], st["dy"].float(), st["rstd"][:, None]
    dn, terms = dy * _weight(st), dy * (xh.to(t).float() if rounded else xh)
    if rounded:
        dn, terms = dn.to(t).float(), terms.to(t).float()
    m = (dn * xh).mean(-1, keepdim=True)
    dx = st["ds"].float() + r * (dn - xh * m)
    return {"dx": dx.to(t), "dw": terms.sum(0).to(st["w"].dtype)}


def _plain(st):
    op, q, group = st["op"], st.get("q"), st.get("group")
    if op == "add":
        s, f, r = _stream(st)
        return {"y": _norm(st, f, r), "s": s, "rstd": r}
    if op == "quant":
        s, f, r = _stream(st)
        y = f * r[:, None] * _weight(st)
        scale = torch.clamp(_groups(y.abs(), group).amax(-1) / QMAX[q], min=FLOOR)
        return {"q": _round8(y / _spread(scale, y.shape[1], group), q), "scale": scale, "s": s}
    if op == "bwd":
        return _gradients(st, st["s"].float() * st["rstd"][:, None], st["variant"] == 0)
    if op == "pack":
        c, scale = _pack(st["x"], q, group)
        return {"c": c, "cscale": scale, "x": (c.float() * _spread(scale, c.shape[1], group)).to(TYPES[st["type"]])}
    if op == "ckpt_fwd":
        s, f, r = _stream(st)
        c, scale = _pack(s, q, group)
        return {"y": _norm(st, f, r), "s": s, "rstd": r, "c": c, "cscale": scale}
    xh = st["c"].float() * _spread(st["cscale"] * st["rstd"][:, None], st["c"].shape[1], group)
    return _gradients(st, xh, False)


# --------------------------------------------------------- the framework's

def _framework(st):
    g, op = _gbn(), st["op"]
    if op == "add":
        y, s, rstd = g.rmsnorm_add_fwd(st["x"], st["res"], st["w"], EPS, variant=st["variant"])
        return {"y": y, "s": s, "rstd": rstd}
    if op == "quant":
        q, scale, s, _ = g.rmsnorm_add_quant_fwd(st["x"], st["res"], st["w"], EPS, Q_TYPES[st["q"]], st["group"],
                                                 save_rstd=False, variant=st["variant"])
        return {"q": q, "scale": scale, "s": s}
    if op == "bwd":
        dx, dw = g.rmsnorm_add_bwd(st["s"], st["dy"], st["w"], st["rstd"], st["ds"], variant=st["variant"])
        return {"dx": dx, "dw": dw}
    if op == "pack":
        c, scale = g.act_pack8(st["x"], Q_TYPES[st["q"]], st["group"])
        return {"c": c, "cscale": scale, "x": g.act_unpack8(c, scale, st["x"].dtype, st["group"])}
    if op == "ckpt_fwd":
        y, s, rstd, c, scale = g.rmsnorm_add_ckpt_fwd(st["x"], st["res"], st["w"], EPS, Q_TYPES[st["q"]], st["group"],
                                                      variant=st["variant"])
        return {"y": y, "s": s, "rstd": rstd, "c": c, "cscale": scale}
    dx, dw = g.rmsnorm_add_ckpt_bwd(st["c"], st["cscale"], st["dy"], st["w"], st["rstd"], st["ds"], st["group"],
                                    variant=st["variant"])
    return {"dx": dx, "dw": dw}


def run(state):
    return _framework(state) if own else _plain(state)


# ------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """run's outputs from the definition in 64 bits.  s (and, in expression 0,
    the normalised value and the backward's products) are held in x's type by
    the definition; an 8-bit value's exact counterpart is the value before
    its rounding."""
    st = prepare(case, seed)
    t, op, N, group = TYPES[case["type"]], case["op"], case["N"], case.get("group", 0)
    d = lambda v: v.to(torch.float64)  # noqa: E731
    held = lambda v: v.to(t).to(torch.float64)  # noqa: E731
    w = d(st["w"]) + (1.0 if case["variant"] == 2 else 0.0)
    width = group or N
    column = torch.arange(N, device="cuda") // width
    count = -(-N // width)

    def scales(v):
        top = torch.zeros(case["M"], count, dtype=torch.float64, device="cuda")
        top.scatter_reduce_(1, column.expand(case["M"], N), v.abs(), "amax")
        return (top / QMAX[case["q"]]).clamp_(min=FLOOR)

    if op == "pack":
        x = d(st["x"])
        sc = scales(x)
        # what is read back follows from the 8-bit values, not from x: no counterpart
        return {"c": x / sc[:, column], "cscale": sc, "x": None}
    if op in ("add", "quant", "ckpt_fwd"):
        total = d(st["x"]) + d(st["res"])
        s = held(total)
        r = (s.square().sum(1) / N + EPS).rsqrt()
        n = s * r[:, None]
        if op == "quant":
            y = n * w
            sc = scales(y)
            return {"q": y / sc[:, column], "scale": sc, "s": total}
        out = {"y": (held(n) if case["variant"] == 0 else n) * w, "s": total, "rstd": r}
        if op == "ckpt_fwd":
            sc = scales(s)
            out.update(c=s / sc[:, column], cscale=sc)
        return out
    r, dy = d(st["rstd"])[:, None], d(st["dy"])
    xh = (d(st["s"]) if op == "bwd" else d(st["c"]) * d(st["cscale"])[:, column]) * r
    dn, terms = dy * w, dy * xh
    if op == "bwd" and case["variant"] == 0:
        dn, terms = held(dn), held(dy * held(xh))
    dx = d(st["ds"]) + r * (dn - xh * ((dn * xh).sum(1, keepdim=True) / N))
    return {"dx": dx, "dw": terms.sum(0)}
