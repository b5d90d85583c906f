"""RMSNorm with the residual's addition, its 8-bit output, the 8-bit
activation checkpoints and their backwards, against the plain 64-bit forms."""
import pytest
import torch

import _addnorm as ref
from normalization_layers_fwd_gb300 import _lib

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
E4, I8 = torch.float8_e4m3fn, torch.int8
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from normalization_layers_fwd_gb300 import build
    build.build()
    _lib.load()
    yield
    assert _lib.read_faults() == 0


def make(M, N, t, wt, variant=1, seed=0):
    """x, residual, w, dy, ds."""
    g = torch.Generator(device="cuda").manual_seed(1000003 * M + 131 * N + seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    w = 0.1 * n(N) + (0.0 if variant == 2 else 1.0)
    gain = torch.where(torch.rand(N, generator=g, device="cuda") < 0.02, 8.0, 1.0)
    return (n(M, N).to(t), (1.5 * n(M, N) * gain).to(t), w.to(wt), (0.1 * n(M, N)).to(t),
            (0.1 * n(M, N)).to(t))


# rows and widths: one of each; below, at and above a vector, a warp's share, a group and the
# schedules' capacities; odd and even widths that are not whole vectors; wider than any schedule
SHAPES = [(1, 1), (3, 2), (5, 7), (2, 8), (70, 24), (129, 31), (40, 32), (33, 33), (300, 64),
          (17, 100), (257, 127), (64, 128), (31, 129), (9, 250), (130, 256), (12, 257),
          (7, 511), (150, 512), (5, 520), (3, 1000), (41, 1001), (160, 1024), (2, 1030), (6, 2048),
          (310, 2050), (1, 4096), (11, 4097), (4, 5001), (33, 8192), (2, 8193), (5, 12001),
          (3, 16384), (2, 16385), (2, 20000)]
TYPES = [(BF, BF, 0), (BF, F32, 1), (F16, F16, 2), (F16, F32, 0), (F32, F32, 1), (BF, BF, 1),
         (F32, BF, 2)]


def pick(i):
    """Every type with every kind of width, over the shapes in turn."""
    return [TYPES[i % len(TYPES)], TYPES[(i + 3) % len(TYPES)]]


CASES = [(M, N, *c) for i, (M, N) in enumerate(SHAPES) for c in pick(i)]


@pytest.mark.parametrize("M,N,t,wt,variant", CASES)
def test_forward(M, N, t, wt, variant):
    x, res, w, _, _ = make(M, N, t, wt, variant)
    y, s, rstd = _lib.rmsnorm_add_fwd(x, res, w, EPS, variant=variant)
    ref.same("s", s, ref.stream(x, res))
    ref.check_rstd(rstd, s, EPS)
    ref.check_y(y, s, w, EPS, variant)
    # without a residual: the norm of x itself
    y, s, rstd = _lib.rmsnorm_add_fwd(x, None, w, EPS, variant=variant)
    assert s is x
    ref.check_rstd(rstd, x, EPS)
    ref.check_y(y, x, w, EPS, variant)


@pytest.mark.parametrize("group,q", [(0, E4), (128, E4), (32, I8), (64, E4), (0, I8)])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_quantised_output(i, group, q):
    (M, N), (t, wt, variant) = SHAPES[i], TYPES[(i + group) % len(TYPES)]
    x, res, w, _, _ = make(M, N, t, wt, variant)
    out, scale, s, rstd = _lib.rmsnorm_add_quant_fwd(x, res, w, EPS, q, group, variant=variant)
    assert out.dtype == q and scale.shape == (M, 1 if group == 0 else -(-N // group))
    ref.same("s", s, ref.stream(x, res))
    ref.check_rstd(rstd, s, EPS)
    ref.check_quant(out, scale, s, w, EPS, variant, group)


@pytest.mark.parametrize("group,q", [(0, E4), (128, I8), (32, E4), (64, I8), (128, E4)])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_checkpoint(i, group, q):
    """The forward's checkpoint and the stand-alone one are the definition's
    bits; reading it back likewise."""
    (M, N), (t, wt, variant) = SHAPES[i], TYPES[(i + group) % len(TYPES)]
    x, res, w, _, _ = make(M, N, t, wt, variant)
    y, s, rstd, c, cscale = _lib.rmsnorm_add_ckpt_fwd(x, res, w, EPS, q, group, variant=variant)
    ref.same("s", s, ref.stream(x, res))
    ref.check_rstd(rstd, s, EPS)
    ref.check_y(y, s, w, EPS, variant)
    c0, cscale0 = ref.pack(s, q, group)
    ref.same("cscale", cscale, cscale0)
    ref.same("c", c, c0)
    c1, cscale1 = _lib.act_pack8(s, q, group)
    ref.same("act_pack8 cscale", cscale1, cscale0)
    ref.same("act_pack8 c", c1, c0)
    for back in (t, F32):
        ref.same("act_unpack8", _lib.act_unpack8(c, cscale, back, group),
                 ref.unpack(c0, cscale0, back, group))


@pytest.mark.parametrize("M,N,t,wt,variant", CASES)
def test_backward(M, N, t, wt, variant):
    x, res, w, dy, ds = make(M, N, t, wt, variant)
    _, s, rstd = _lib.rmsnorm_add_fwd(x, res, w, EPS, variant=variant)
    xh = ref.d(s) * ref.d(rstd)[:, None]
    for d_s in (ds, None):
        dx, dw = _lib.rmsnorm_add_bwd(s, dy, w, rstd, d_s, variant=variant)
        ref.check_gradients(dx, dw, xh, dy, d_s, w, rstd, variant, variant == 0)
    dx2, none = _lib.rmsnorm_add_bwd(s, dy, w, rstd, None, need_dw=False, variant=variant)
    assert none is None
    ref.same("dx without dw", dx2, dx)


@pytest.mark.parametrize("group,q", [(0, E4), (128, I8), (32, E4), (64, I8), (128, E4)])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_backward_from_checkpoint(i, group, q):
    (M, N), (t, wt, variant) = SHAPES[i], TYPES[(i + group) % len(TYPES)]
    x, res, w, dy, ds = make(M, N, t, wt, variant)
    _, s, rstd, c, cscale = _lib.rmsnorm_add_ckpt_fwd(x, res, w, EPS, q, group, variant=variant)
    xh = (ref.d(c.float()) * ref.spread(ref.d(cscale), N, group) * ref.d(rstd)[:, None])
    for d_s in (ds, None):
        dx, dw = _lib.rmsnorm_add_ckpt_bwd(c, cscale, dy, w, rstd, d_s, group, variant=variant)
        ref.check_gradients(dx, dw, xh, dy, d_s, w, rstd, variant, False)


@pytest.mark.parametrize("N", [64, 129, 1024, 2050])
@pytest.mark.parametrize("variant", [1, 2])
def test_gradient_against_differences(N, variant):
    """The float32 kernels' gradients of a random linear reading of y and s,
    against central differences of the 64-bit formula along random directions.
    Differences: h = 1e-5 leaves an h^2 term near 1e-9; the kernels' dx and dw
    are within 1e-4 of their size by test_backward's bounds, and a direction
    adds M N of them."""
    M = 6
    x, res, w, dy, ds = make(M, N, F32, F32, variant, seed=5)
    _, s, rstd = _lib.rmsnorm_add_fwd(x, res, w, EPS, variant=variant)
    dx, dw = _lib.rmsnorm_add_bwd(s, dy, w, rstd, ds, variant=variant)

    def loss(s64, w64):
        y = s64 * (s64.square().mean(-1, keepdim=True) + EPS).rsqrt() * (
            w64 + (1.0 if variant == 2 else 0.0))
        return (y * ref.d(dy)).sum() + (s64 * ref.d(ds)).sum()

    g = torch.Generator(device="cuda").manual_seed(9)
    vs = torch.randn(M, N, generator=g, device="cuda", dtype=torch.float64)
    vw = torch.randn(N, generator=g, device="cuda", dtype=torch.float64)
    h = 1e-5
    num = (loss(ref.d(s) + h * vs, ref.d(w) + h * vw)
           - loss(ref.d(s) - h * vs, ref.d(w) - h * vw)) / (2 * h)
    terms = torch.cat([(ref.d(dx) * vs).reshape(-1), ref.d(dw) * vw])
    assert abs(float(num - terms.sum())) <= 1e-5 * float(terms.abs().sum()) + 1e-7


# ------------------------------------------------------------ strides, aliases

def views(M, N, t, seed):
    """The same kind of rows in other places: a slice of wider rows, a column
    slice that is not on a vector boundary, every second row, a broadcast row."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda").to(t)  # noqa: E731
    return {"padded": n(M, N + 16)[:, :N], "odd": n(M, N + 3)[:, 1:N + 1], "second": n(2 * M, N)[::2],
            "broadcast": n(1, N).expand(M, N)}


@pytest.mark.parametrize("N", [128, 1024, 1001, 2056])
@pytest.mark.parametrize("t", [BF, F32])
def test_strided_inputs(N, t):
    """Strided x, residual, s, dy and ds give the bits of their copies."""
    M = 32
    _, _, w, _, _ = make(M, N, t, t)
    a, b = views(M, N, t, 1), views(M, N, t, 2)
    for (ka, x), (kb, res) in zip(a.items(), list(b.items())[1:] + list(b.items())[:1]):
        y, s, rstd = _lib.rmsnorm_add_fwd(x, res, w, EPS, variant=1)
        ref.same(f"s {ka} {kb}", s, ref.stream(x, res))
        ref.check_rstd(rstd, s, EPS)
        ref.check_y(y, s, w, EPS, 1)
        q, scale, s2, _ = _lib.rmsnorm_add_quant_fwd(x, res, w, EPS, E4, 64, variant=1)
        ref.same("s", s2, s)
        ref.check_quant(q, scale, s, w, EPS, 1, 64)
        c, cscale = _lib.act_pack8(x, I8, 128)
        c0, cscale0 = ref.pack(x.contiguous(), I8, 128)
        ref.same("c", c, c0)
        ref.same("cscale", cscale, cscale0)
        r = ref.rstd_of(x, EPS).float()
        dx, dw = _lib.rmsnorm_add_bwd(x, res, w, r, a["padded"], variant=1)
        ref.check_gradients(dx, dw, ref.d(x) * ref.d(r)[:, None], res, a["padded"], w, r, 1, False)


def test_head_major_and_leading_dimensions():
    """[B, H, S, D] seen as [B, S, H, D]: outputs keep the leading shape."""
    B, H, S, D = 2, 4, 9, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(B, H, S, D, generator=g, device="cuda").to(BF).transpose(1, 2)
    res = torch.randn(B, S, H, D, generator=g, device="cuda").to(BF)
    w = torch.ones(D, device="cuda")
    y, s, rstd, c, cscale = _lib.rmsnorm_add_ckpt_fwd(x, res, w, EPS, E4, 32, variant=1)
    assert y.shape == s.shape == c.shape == (B, S, H, D) and cscale.shape == (B, S, H, 4)
    ref.same("s", s, ref.stream(x, res))
    ref.check_y(y, s, w, EPS, 1)
    dx, dw = _lib.rmsnorm_add_ckpt_bwd(c, cscale, x, w, rstd, res, 32, variant=1)
    assert dx.shape == (B, S, H, D)
    xh = (ref.d(c.float()).reshape(-1, D) * ref.spread(ref.d(cscale), D, 32)
          * ref.d(rstd)[:, None])
    ref.check_gradients(dx, dw, xh, x, res, w, rstd, 1, False)


@pytest.mark.parametrize("M,N", [(5, 4096), (37, 1001), (300, 64), (2, 20000), (3, 8191)])
def test_update_in_place(M, N):
    """The stream may take the place of the residual, or of x."""
    x, res, w, _, _ = make(M, N, BF, BF)
    y0, s0, r0 = _lib.rmsnorm_add_fwd(x, res, w, EPS, variant=1)
    q0, sc0, _, _ = _lib.rmsnorm_add_quant_fwd(x, res, w, EPS, E4, 128, variant=1)
    for which in (0, 1):
        a, b = x.clone(), res.clone()
        y, s, r = _lib.rmsnorm_add_fwd(a, b, w, EPS, variant=1, s=(a, b)[which])
        assert s is (a, b)[which]
        ref.same("s", s, s0), ref.same("y", y, y0), ref.same("rstd", r, r0)
        a, b = x.clone(), res.clone()
        q, sc, s, _ = _lib.rmsnorm_add_quant_fwd(a, b, w, EPS, E4, 128, variant=1,
                                                 s=(a, b)[which])
        ref.same("s", s, s0), ref.same("q", q, q0), ref.same("scale", sc, sc0)


# ----------------------------------------------------- values that are special

@pytest.mark.parametrize("N", [64, 1001, 4096])
def test_zero_rows(N):
    x = torch.zeros(3, N, device="cuda", dtype=BF)
    w = torch.ones(N, device="cuda")
    y, s, rstd, c, cscale = _lib.rmsnorm_add_ckpt_fwd(x, x, w, EPS, E4, 32)
    assert torch.all(y == 0) and torch.all(s == 0) and torch.all(c.float() == 0)
    assert torch.all(cscale == ref.FLOOR)
    q, scale, _, _ = _lib.rmsnorm_add_quant_fwd(x, x, w, EPS, I8, 0)
    assert torch.all(q == 0) and torch.all(scale == ref.FLOOR)
    dx, dw = _lib.rmsnorm_add_ckpt_bwd(c, cscale, torch.ones_like(x), w, rstd, None, 32)
    assert torch.all(dw == 0) and torch.all(torch.isfinite(dx))


@pytest.mark.parametrize("N,group", [(256, 32), (1001, 128), (1001, 0), (4096, 64), (20000, 128)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("q", [E4, I8])
def test_non_finite_values(N, group, bad, q):
    """A group with a NaN or an infinity reads back as NaN throughout; other
    groups and rows are untouched.  A norm's row with one has rstd NaN or 0."""
    x, res, w, _, _ = make(4, N, BF, BF)
    clean = _lib.act_pack8(x, q, group)
    y0, _, _, = _lib.rmsnorm_add_fwd(x, res, w, EPS, variant=1)
    col = N - 3
    x[1, col] = bad
    c, cscale = _lib.act_pack8(x, q, group)
    v = _lib.act_unpack8(c, cscale, F32, group)
    g = group or N
    inside = torch.zeros(4, N, dtype=torch.bool, device="cuda")
    inside[1, col // g * g:min(col // g * g + g, N)] = True
    assert torch.equal(torch.isnan(v), inside)
    ref.same("other groups", c[~inside], clean[0][~inside])
    out, scale, s, rstd = _lib.rmsnorm_add_quant_fwd(x, res, w, EPS, q, group, variant=1)
    y, s, rstd = _lib.rmsnorm_add_fwd(x, res, w, EPS, variant=1)
    dq = _lib.act_unpack8(out, scale, F32, group)
    assert torch.isfinite(dq[[0, 2, 3]]).all() and torch.isfinite(rstd[[0, 2, 3]]).all()
    ref.same("other rows", y[[0, 2, 3]], y0[[0, 2, 3]])
    if bad != bad:
        assert torch.isnan(rstd[1]) and torch.isnan(y[1]).all() and torch.isnan(dq[1]).all()
    else:  # r = 0: zero beside the infinity, NaN at it (its group in 8 bits)
        assert rstd[1] == 0 and torch.isnan(y[1, col]) and torch.isnan(dq[1])[inside[1]].all()
        assert torch.all(dq[1][~inside[1]] == 0)


def test_magnitudes():
    """Rows from 2^-60 to 2^60 in float32: scales follow, nothing saturates."""
    N = 512
    base, _, w, _, _ = make(121, N, F32, F32)
    x = base * torch.exp2(torch.arange(-60, 61, device="cuda", dtype=F32))[:, None]
    for q in (E4, I8):
        c, cscale = _lib.act_pack8(x, q, 64)
        c0, s0 = ref.pack(x, q, 64)
        ref.same("c", c, c0)
        ref.same("cscale", cscale, s0)
    # eps is far above the smallest rows' squares and far below the largest's.  A row whose sum
    # of squares passes 2^128 is outside float32: r is rsqrt(inf) = 0 there and y with it, as in
    # rmsnorm_fwd.  (512 squares of about 2^120: the last row's sum is about 2^129.)
    y, s, rstd = _lib.rmsnorm_add_fwd(x, torch.zeros_like(x), w, EPS, variant=1)
    over = ref.d(s).square().sum(-1) >= 2.0 ** 128
    assert 0 < int(over.sum()) <= 1
    assert torch.all(rstd[over] == 0) and torch.all(y[over] == 0)
    ref.check_y(y[~over], s[~over], w, EPS, 1)


def test_empty_input():
    for N in (8, 33):
        x = torch.empty(0, N, device="cuda", dtype=BF)
        w = torch.ones(N, device="cuda")
        y, s, rstd = _lib.rmsnorm_add_fwd(x, x, w)
        assert y.shape == (0, N) and rstd.shape == (0,)
        q, scale, _, _ = _lib.rmsnorm_add_quant_fwd(x, x, w, group=32)
        dx, dw = _lib.rmsnorm_add_bwd(x, x, w, rstd)
        assert dx.shape == (0, N) and torch.all(dw == 0)
        c, cscale = _lib.act_pack8(x)
        assert _lib.act_unpack8(c, cscale).shape == (0, N)
