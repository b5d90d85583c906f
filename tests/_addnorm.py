"""Plain 64-bit forms of the residual-stream operators, and how far the
kernels' outputs may be from them.

Tolerances, from the kernels' arithmetic.  u = 2^-24 is half a step of
float32, h half a step of an output's type (2^-9 bf16, 2^-12 fp16 relative to
a binade's lower end, so eps / 2 of torch.finfo: 2^-8 and 2^-11 of a value at
worst; 2^-24 for float32).

* A float32 sum of N products over a row takes at most N / 32 + 16 additions
  in a row (a lane's share at 32 lanes, then the tree), each off by u of the
  partial sum: chain(N) = N / 32 + 20 steps with the products' own roundings.
* r = rsqrt(sum / N + eps): half the sum's relative error, and 2 ulp = 4u of
  the function: within chain(N) u + 8u.
* y = w' s r: two more products (2u) and one rounding (h); expression 0
  rounds twice (2h).
* The 8-bit values: half a step of the type, relative 2^-4 or 2^-10 of the
  scale in e4m3's subnormals, half the scale in int8; the float32 value in
  front of that rounding is off by r's error and 8u.
* dx = ds + r (dn - xh m): each of the three terms carries a few u, and m the
  chain of its sum; then h.  dw: M terms added one after another at worst.
"""
import torch

U = 2.0 ** -24
FLOOR = 2.0 ** -100
QMAX = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}


def half(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    """The smallest subnormal of a type."""
    return torch.finfo(t).tiny * torch.finfo(t).eps


def chain(N):
    return N / 32 + 20


def d(v):
    return v.to(torch.float64)


def weight(w, variant):
    return d(w) + (1.0 if variant == 2 else 0.0)


def close(name, got, want, tol):
    """|got - want| <= tol everywhere, NaN and infinities in the same places."""
    got, want = d(got).reshape(-1), d(want).reshape(-1)
    tol = torch.as_tensor(tol, dtype=torch.float64, device=got.device).expand(
        want.shape if torch.as_tensor(tol).dim() == 0 else tol.shape).reshape(-1)
    assert got.shape == want.shape, name
    fine = torch.isfinite(want)
    assert torch.equal(fine, torch.isfinite(got)), f"{name}: non-finite values in other places"
    assert torch.equal(torch.isnan(want), torch.isnan(got)), f"{name}: NaN in other places"
    bad = fine & ((got - want).abs() > tol)
    if bad.any():
        i = int(bad.nonzero()[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off; first at {i}: "
                             f"{float(got[i])!r}, want {float(want[i])!r} +- {float(tol[i]):.3g}")


def stream(x, res):
    """The stream, in x's type: one float32 addition, one rounding."""
    return x if res is None else (x.float() + res.float()).to(x.dtype)


def rstd_of(s, eps):
    return (d(s).square().mean(-1) + eps).rsqrt()


def check_rstd(rstd, s, eps):
    want = rstd_of(s, eps)
    close("rstd", rstd.view(want.shape), want, want * (chain(s.shape[-1]) + 8) * U)


def check_y(y, s, w, eps, variant):
    t, N = s.dtype, s.shape[-1]
    want = d(s) * rstd_of(s, eps)[..., None] * weight(w, variant)
    roundings = 2 if variant == 0 else 1
    rel = (1 + half(t)) ** roundings - 1 + (chain(N) + 12) * U
    big = 2 + weight(w, variant).abs()
    close("y", y, want, want.abs() * rel * (1 + 2 * half(t)) + big * tiny(t))


def groups(v, group):
    """v [..., N] as [rows, groups, columns], filled up with zeros."""
    N = v.shape[-1]
    g = group or N
    n = -(-N // g)
    v = v.reshape(-1, N)
    return torch.nn.functional.pad(v, (0, n * g - N)).view(-1, n, g)


def spread(scale, N, group):
    scale = scale.reshape(-1, scale.shape[-1])
    return scale.expand(-1, N) if group == 0 else scale.repeat_interleave(group, 1)[:, :N]


def pack(x, dtype, group):
    """act_pack8's definition, step for step in float32."""
    f = x.float().reshape(-1, x.shape[-1])
    amax = groups(f.abs(), group).amax(-1)
    scale = torch.maximum(amax * torch.tensor(1.0 / QMAX[dtype], dtype=torch.float32,
                                              device=x.device),
                          torch.tensor(FLOOR, dtype=torch.float32, device=x.device))
    v = f * spread(1.0 / scale, f.shape[1], group)
    q = v.to(dtype) if dtype == torch.float8_e4m3fn else v.round().to(dtype)
    return q.view(x.shape), scale.view(*x.shape[:-1], -1)


def unpack(c, cscale, dtype, group):
    v = c.float().reshape(-1, c.shape[-1]) * spread(cscale, c.shape[-1], group)
    return v.to(dtype).view(c.shape)


def bits(t):
    return t.contiguous().view({1: torch.int8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def same(name, a, b):
    assert a.shape == b.shape and a.dtype == b.dtype, name
    assert torch.equal(bits(a), bits(b)), f"{name}: {int((bits(a) != bits(b)).sum())} differ"


def check_quant(q, scale, s, w, eps, variant, group):
    N = s.shape[-1]
    y = (d(s) * rstd_of(s, eps)[..., None] * weight(w, variant)).reshape(-1, N)
    want = torch.clamp(groups(y.abs(), group).amax(-1) / QMAX[q.dtype], min=FLOOR)
    err = (chain(N) + 16) * U
    close("scale", scale.reshape(want.shape), want, want * err)
    sc = spread(d(scale), N, group)
    step = (torch.maximum(y.abs() * 2.0 ** -4, sc * 2.0 ** -10) if q.dtype == torch.float8_e4m3fn
            else sc / 2)
    close("q * scale", q.reshape(-1, N).to(torch.float32).double() * sc, y,
          step * (1 + 4 * err) + y.abs() * err)


def gradients(xh, dy, ds, w, rstd, variant, rounded):
    """dx and dw in 64 bits (rounded: expression 0's rounding points), and what
    their tolerances are made of."""
    t, N = dy.dtype, dy.shape[-1]
    dy64, r = d(dy).reshape(-1, N), d(rstd).reshape(-1, 1)
    xh = xh.reshape(-1, N)
    dn, terms = dy64 * weight(w, variant), dy64 * xh
    if rounded:
        dn = dn.to(t).double()
        terms = dy64 * xh.to(t).double()
        if w.dtype != torch.float32:
            terms = terms.to(t).double()
    m = (dn * xh).mean(-1, keepdim=True)
    ds64 = torch.zeros_like(dn) if ds is None else d(ds).reshape(-1, N)
    dx = ds64 + r * (dn - xh * m)
    return dx, terms, dn, m, ds64, r


def check_gradients(dx, dw, xh, dy, ds, w, rstd, variant, rounded):
    t, N = dy.dtype, dy.shape[-1]
    M = dy.numel() // N
    xh = xh.reshape(-1, N)
    want, terms, dn, m, ds64, r = gradients(xh, dy, ds, w, rstd, variant, rounded)
    size = ds64.abs() + r * (dn.abs() + (xh * m).abs())
    mean_err = (dn * xh).abs().mean(-1, keepdim=True) * (chain(N) + 4) * U
    tol = want.abs() * half(t) + size * (8 * U) * (1 + half(t)) + r * xh.abs() * mean_err + tiny(t)
    if rounded and w.dtype == torch.float32 and t != torch.float32:
        # dy w is rounded to float32 before x's type: next to a border it may go the other way
        tol = tol + 2 * half(t) * (r * dn.abs() + r * xh.abs()
                                   * (dn * xh).abs().mean(-1, keepdim=True))
    close("dx", dx, want, tol)
    if dw is None:
        return
    total = terms.sum(0)
    tol = total.abs() * half(dw.dtype) + terms.abs().sum(0) * ((M + 4) * U) + tiny(dw.dtype)
    if rounded and t != torch.float32:
        # xhat's float32 error may turn a rounding of xhat (and then of its term) next to a
        # border: 2^-15 of the values at most, so four of a column's few hundred terms
        tol = tol + 4 * 4 * half(t) * terms.abs().amax(0)
    close("dw", dw, total, tol)
