"""The residual-stream operators as a program uses them: through autograd,
several layers together, captured into graphs, on several streams, on large
tensors, next to memory that is not theirs."""
import ctypes

import pytest
import torch

import _addnorm as ref
from normalization_layers_fwd_gb300 import _lib
from normalization_layers_fwd_gb300 import functional as F

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def plain_norm(s, w):
    return s * (s.square().mean(-1, keepdim=True) + EPS).rsqrt() * w


def stack(x, res, ws, mats, norm):
    """Three blocks: the stream takes each block's output in and feeds the next."""
    for w, m in zip(ws, mats):
        y, res = norm(x, res, w)
        x = y @ m
    return x.square().sum() + 0.5 * res.square().sum()


@pytest.mark.parametrize("N", [96, 129, 512])
@pytest.mark.parametrize("checkpoint", [None, E4, I8])
def test_layers_together(N, checkpoint):
    """Gradients of a stack of three blocks in float32 against the same stack
    in float64.  Without a checkpoint they differ by float32 rounding, which
    three blocks of products of N terms leave below 1e-4 of the gradients'
    size; an 8-bit stream is off by 2^-4 (e4m3) or 1/254 of its group's
    largest (int8) per element, at random, so the gradients by less than
    twice that."""
    g = gen(N)
    M = 24
    x, res = randn(g, 2, M, N), randn(g, 2, M, N)
    ws = [1 + 0.1 * randn(g, N) for _ in range(3)]
    mats = [randn(g, N, N) / N ** 0.5 for _ in range(3)]
    leaves = [t.clone().requires_grad_() for t in (x, res, *ws)]
    loss = stack(leaves[0], leaves[1], leaves[2:], mats,
                 lambda a, b, w: F.add_rms_norm(a, b, w, EPS, 1, checkpoint, 32))
    got = torch.autograd.grad(loss, leaves)
    exact = [t.double().requires_grad_() for t in (x, res, *ws)]
    loss64 = stack(exact[0], exact[1], exact[2:], [m.double() for m in mats],
                   lambda a, b, w: (plain_norm(a + b, w), a + b))
    want = torch.autograd.grad(loss64, exact)
    assert abs(float(loss.detach()) / float(loss64.detach()) - 1) < 1e-4
    far = {None: 1e-4, E4: 2 * 2 ** -4, I8: 2 * 3.0 / 254 * 2}[checkpoint]
    for a, b in zip(got, want):
        assert a.shape == b.shape
        assert float((a.double() - b).norm() / b.norm()) < far


def test_gradient_paths():
    """Gradients where only y, only s, or neither of x and residual needs one;
    the same tensor twice; a broadcast residual."""
    g = gen(1)
    x, res, w = randn(g, 6, 64), randn(g, 6, 64), 1 + 0.1 * randn(g, 64)
    dy = randn(g, 6, 64)

    def grads(fn, *leaves):
        leaves = [t.clone().requires_grad_() for t in leaves]
        return torch.autograd.grad(fn(*leaves), leaves)

    def plain(a, b, c):
        return plain_norm(a.double() + b.double(), c.double())

    def mine(a, b, c):
        return F.add_rms_norm(a, b, c, EPS, 1)[0]

    cases = [
        (lambda f: lambda a, b, c: (f(a, b, c) * dy).sum(), (x, res, w)),
        (lambda f: lambda a: (f(a, a, w) * dy).sum(), (x,)),
        (lambda f: lambda a, b: (f(a, b.expand(6, 64), w) * dy).sum(), (x, res[:1])),
        (lambda f: lambda c: (f(x, res, c) * dy).sum(), (w,)),
    ]
    for make, leaves in cases:
        for a, b in zip(grads(make(mine), *leaves), grads(make(plain), *leaves)):
            ref.close("gradient", a, b, 1e-5 * float(b.abs().max()))
    # only s is used: the norm passes nothing back
    a, b = x.clone().requires_grad_(), res.clone().requires_grad_()
    c = w.clone().requires_grad_()
    s = F.add_rms_norm(a, b, c, EPS, 1)[1]
    da, db, dc = torch.autograd.grad((s * dy).sum(), (a, b, c), allow_unused=True)
    ref.same("ds", da, dy), ref.same("ds", db, dy)
    assert dc is None


@pytest.mark.parametrize("checkpoint", [E4, I8])
def test_checkpointed_layers(checkpoint):
    """dyt, layer_norm and rms_norm from a checkpoint: the gradients of the
    unpacked input, with the forward's own statistics."""
    g = gen(2)
    N = 200
    x, dy = randn(g, 3, 7, N, dtype=BF), randn(g, 3, 7, N, dtype=BF)
    p, b, a = 1 + 0.1 * randn(g, N), randn(g, N), torch.full((1,), 0.7, device="cuda")
    back = _lib.act_unpack8(*_lib.act_pack8(x, checkpoint, 64), BF, 64)

    def grads(fn):
        xl, pl = x.clone().requires_grad_(), p.clone().requires_grad_()
        return torch.autograd.grad(fn(xl, pl), (xl, pl), dy)

    dx, dp = grads(lambda t, q: F.dyt(t, a, q, b, checkpoint, 64))
    ex, _, eg, _ = _lib.dyt_bwd(back, dy, a, p)
    ref.same("dyt dx", dx, ex.view_as(dx)), ref.same("dyt dgamma", dp, eg)
    dx, dp = grads(lambda t, q: F.layer_norm(t, q, b, 1e-5, checkpoint, 64))
    _, mean, rstd = _lib.layernorm_fwd(x, p, b, 1e-5)
    ex, eg, _ = _lib.layernorm_bwd(back, dy, mean, rstd, p)
    ref.same("ln dx", dx, ex.view_as(dx)), ref.same("ln dgamma", dp, eg)
    dx, dp = grads(lambda t, q: F.rms_norm(t, q, EPS, 1, checkpoint, 64))
    _, rstd = _lib.rmsnorm_fwd(x, p, EPS, variant=1)
    c, sc = _lib.act_pack8(x, checkpoint, 64)
    xh = ref.d(c.float()).reshape(-1, N) * ref.spread(ref.d(sc), N, 64) * ref.d(rstd)[:, None]
    ref.check_gradients(dx, dp, xh, dy, None, p, rstd, 1, False)


def test_quantised_output_refuses_gradients():
    x = torch.zeros(2, 64, device="cuda", requires_grad=True)
    w = torch.ones(64, device="cuda")
    with pytest.raises(RuntimeError, match="no gradient"):
        F.add_rms_norm_quant(x, x, w)
    with torch.no_grad():
        q, scale, s = F.add_rms_norm_quant(x, x, w)
    assert q.dtype == E4 and scale.shape == (2, 1) and s.shape == (2, 64)


def test_bindings_refuse():
    x = torch.zeros(4, 64, device="cuda", dtype=BF)
    w = torch.ones(64, device="cuda")
    r = torch.ones(4, device="cuda")
    c, sc = _lib.act_pack8(x, E4, 32)
    for bad in (lambda: _lib.rmsnorm_add_fwd(x, x[:3], w),
                lambda: _lib.rmsnorm_add_fwd(x, x.float(), w),
                lambda: _lib.rmsnorm_add_fwd(x, x.cpu(), w),
                lambda: _lib.rmsnorm_add_fwd(x, x, w[:63]),
                lambda: _lib.rmsnorm_add_fwd(x, None, w, s=x.clone()),
                lambda: _lib.rmsnorm_add_fwd(x, x, w, s=torch.zeros(4, 80, device="cuda",
                                                                    dtype=BF)[:, :64]),
                lambda: _lib.rmsnorm_add_quant_fwd(x, x, w, group=16),
                lambda: _lib.act_pack8(x, E4, -1),
                lambda: _lib.act_unpack8(c, sc[:, :1], BF, 32),
                lambda: _lib.act_unpack8(c, sc, BF, 64),
                lambda: _lib.act_unpack8(c, sc.half(), BF, 32),
                lambda: _lib.rmsnorm_add_ckpt_bwd(c[:3], sc, x, w, r, group=32),
                lambda: _lib.rmsnorm_add_bwd(x, x, w, r[:3]),
                lambda: _lib.rmsnorm_add_bwd(x, x, w, r, x[:, :32])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: _lib.rmsnorm_add_fwd(x.int(), x.int(), w),
                lambda: _lib.act_unpack8(x, sc, BF, 32),
                lambda: _lib.act_unpack8(c, sc, torch.float64, 32),
                lambda: _lib.rmsnorm_add_bwd(x, x, w, r.half())):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(_lib.GbnError, match="GBN_EINVAL"):
        _lib.rmsnorm_add_fwd(x, x, w, eps=-1.0)
    with pytest.raises(_lib.GbnError, match="GBN_EINVAL"):
        _lib.rmsnorm_add_fwd(x, x, w, variant=3)
    with pytest.raises(_lib.GbnError, match="GBN_EDTYPE"):
        _lib.rmsnorm_add_fwd(x, x, w.half())


# -------------------------------------------------------- graphs and streams

def every_call(x, res, w, dy, ds):
    """One of each, as tensors."""
    y, s, rstd = _lib.rmsnorm_add_fwd(x, res, w, EPS, variant=1)
    q, sc, _, _ = _lib.rmsnorm_add_quant_fwd(x, res, w, EPS, E4, 64)
    _, _, _, c, cs = _lib.rmsnorm_add_ckpt_fwd(x, res, w, EPS, I8, 32)
    a = _lib.rmsnorm_add_bwd(s, dy, w, rstd, ds, variant=1)
    b = _lib.rmsnorm_add_ckpt_bwd(c, cs, dy, w, rstd, ds, 32)
    p = _lib.act_pack8(x, E4, 128)
    return [y, s, rstd, q, sc, c, cs, *a, *b, *p, _lib.act_unpack8(*p, x.dtype, 128)]


def inputs(seed, M, N):
    g = gen(seed)
    return (randn(g, M, N, dtype=BF), randn(g, M, N, dtype=BF), 1 + 0.1 * randn(g, N),
            randn(g, M, N, dtype=BF), randn(g, M, N, dtype=BF))


@pytest.mark.parametrize("M,N", [(5, 129), (700, 512), (1300, 2050)])
def test_reruns_are_identical(M, N):
    t = inputs(3, M, N)
    first = every_call(*t)
    for _ in range(3):
        for a, b in zip(first, every_call(*t)):
            ref.same("rerun", a, b)


def test_two_graphs_replayed_together():
    """Two captures from one stream, replayed at once on two others with new
    inputs: nothing is shared between them."""
    shapes = [(900, 1024), (900, 1024)]
    static = [inputs(10 + i, *s) for i, s in enumerate(shapes)]
    graphs, outs = [], []
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for t in static:
            every_call(*t)
    torch.cuda.synchronize()
    for t in static:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(every_call(*t))
        graphs.append(g)
    for rep in range(3):
        new = [inputs(20 + 2 * rep + i, *s) for i, s in enumerate(shapes)]
        for t, n in zip(static, new):
            for a, b in zip(t, n):
                a.copy_(b)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for t, o in zip(new, outs):
            for a, b in zip(every_call(*t), o):
                ref.same("replay", a, b)


def test_calls_on_two_streams():
    sets = [inputs(30 + i, 600, 1001) for i in range(2)]
    want = [every_call(*t) for t in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(4):
        got = []
        for s, t in zip(streams, sets):
            with torch.cuda.stream(s):
                got.append(every_call(*t))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            for u, v in zip(a, b):
                ref.same("stream", u, v)


def test_training_step_in_a_graph():
    """Forward and backward of a block captured whole, weights updated between
    replays."""
    N = 256
    g = gen(5)
    x, res, dy = (randn(g, 64, N, dtype=BF) for _ in range(3))
    w = (1 + 0.1 * randn(g, N)).requires_grad_()

    def step():
        a, b = x.detach().requires_grad_(), res.detach().requires_grad_()
        y, s = F.add_rms_norm(a, b, w, EPS, 1, E4, 32)
        return torch.autograd.grad((y * dy).float().sum() + s.float().sum(), (a, b, w))

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step()
    for _ in range(2):
        with torch.no_grad():
            w.mul_(1.01)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for a, b in zip(got, step()):
            ref.same("graph", a, b)


# ----------------------------------------------- memory that is not theirs

def guarded(shape, dtype, lead=64):
    """A tensor between two guards, and how to check them (lead: elements of
    guard in front, so its alignment is lead's)."""
    n = 1
    for v in shape:
        n *= v
    buf = torch.full((n + lead + 64,), 1, dtype=torch.int8 if dtype in (E4, I8) else dtype,
                     device="cuda")
    before = buf.clone()
    t = buf[lead:lead + n].view(dtype if dtype in (E4, I8) else dtype).view(shape)

    def check(name):
        assert torch.equal(buf[:lead], before[:lead]), f"{name}: written in front"
        assert torch.equal(buf[lead + n:], before[lead + n:]), f"{name}: written behind"
    return t, check


@pytest.mark.parametrize("M,N", [(1, 1), (3, 33), (130, 65), (9, 1000), (7, 1001), (2, 4097),
                                 (310, 2050), (3, 8200), (2, 16384), (2, 20000)])
@pytest.mark.parametrize("lead", [64, 3])
def test_nothing_is_written_outside(M, N, lead):
    lib = _lib.load()
    x, res, w, dy, ds = inputs(40, M, N)
    st = torch.cuda.current_stream().cuda_stream
    ng = -(-N // 32)
    outs = {}

    def out(name, shape, dtype):
        t, check = guarded(shape, dtype, lead)
        outs[name] = check
        return t, ctypes.c_void_p(t.data_ptr())

    s, ps = out("s", (M, N), BF)
    y, py = out("y", (M, N), BF)
    rstd, pr = out("rstd", (M,), F32)
    c, pc = out("c", (M, N), E4)
    cs, pcs = out("cscale", (M, ng), F32)
    q, pq = out("q", (M, N), I8)
    qs, pqs = out("qscale", (M, ng), F32)
    dx, pdx = out("dx", (M, N), BF)
    dw, pdw = out("dw", (N,), F32)
    x2, px2 = out("x", (M, N), BF)
    n = lib.gbn_bwd_workspace_bytes(3, M, N, 1, 0, 0)
    ws, pws = out("ws", (n // 4,), F32)
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    assert lib.rmsnorm_add_ckpt_fwd(p(x), None, p(res), None, p(w), ps, py, pr, pc, pcs, M, N, 32,
                                    EPS, 1, 0, 8, 1, st) == 0
    assert lib.rmsnorm_add_quant_fwd(p(x), None, p(res), None, p(w), ps, pq, pqs, pr, M, N, 32,
                                     EPS, 1, 0, 9, 1, st) == 0
    assert lib.rmsnorm_add_fwd(p(x), None, p(res), None, p(w), ps, py, pr, M, N, EPS, 1, 0, 1,
                               st) == 0
    assert lib.rmsnorm_add_bwd(ps, None, p(dy), None, p(ds), None, p(w), pr, pdx, pdw, M, N, 1, 0,
                               1, pws, n, st) == 0
    xh = ref.d(s) * ref.d(rstd)[:, None]
    ref.check_gradients(dx, dw, xh, dy, ds, w, rstd, 1, False)
    assert lib.rmsnorm_add_ckpt_bwd(pc, pcs, p(dy), None, p(ds), None, p(w), pr, pdx, pdw, M, N,
                                    32, 1, 0, 8, 1, pws, n, st) == 0
    assert lib.act_pack8(p(x), None, pc, pcs, M, N, 32, 1, 8, st) == 0
    assert lib.act_unpack8(pc, pcs, px2, M, N, 32, 1, 8, st) == 0
    torch.cuda.synchronize()
    for name, check in outs.items():
        check(name)
    ref.same("s", s, ref.stream(x, res))
    ref.check_y(y, s, w, EPS, 1)
    ref.check_quant(q, qs, s, w, EPS, 1, 32)
    c0, cs0 = ref.pack(x, E4, 32)
    ref.same("c", c, c0), ref.same("cscale", cs, cs0)
    ref.same("x", x2, ref.unpack(c0, cs0, BF, 32))


def test_a_small_workspace_is_refused():
    lib = _lib.load()
    x, res, w, dy, ds = inputs(41, 300, 512)
    r = torch.ones(300, device="cuda")
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    need = lib.gbn_bwd_workspace_bytes(3, 300, 512, 1, 0, 0)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    call = lambda n: lib.rmsnorm_add_bwd(p(x), None, p(dy), None, None, None, p(w), p(r), p(dx),  # noqa: E731
                                         p(dw), 300, 512, 1, 0, 1, p(ws), n,
                                         torch.cuda.current_stream().cuda_stream)
    assert call(need) == 0 and call(16) == 3


def test_offsets_past_32_bits():
    """[300000, 8191] has 2.46e9 elements: the last rows against a call of
    their own."""
    M, N, tail = 300000, 8191, 40
    free, _ = torch.cuda.mem_get_info()
    if free < 60 << 30:
        pytest.skip("needs 60 GB")
    x = torch.zeros(M, N, dtype=BF, device="cuda")
    g = gen(6)
    x[-tail:] = randn(g, tail, N, dtype=BF)
    w = 1 + 0.1 * randn(g, N)
    small = x[-tail:].clone()
    y, s, rstd, c, cs = _lib.rmsnorm_add_ckpt_fwd(x, x, w, EPS, E4, 64, variant=1)
    a = _lib.rmsnorm_add_ckpt_fwd(small, small, w, EPS, E4, 64, variant=1)
    for big, one in zip((y, s, rstd, c, cs), a):
        assert torch.allclose(big[-tail:].float(), one.float(), rtol=2e-2, atol=1e-6)
    ref.same("s", s[-tail:], a[1])
    ref.same("c", c[-tail:], a[3])
    ref.check_y(y[-tail:], s[-tail:], w, EPS, 1)
    ref.same("unpack", _lib.act_unpack8(c, cs, BF, 64)[-tail:],
             _lib.act_unpack8(a[3], a[4], BF, 64))
    del y, x
    dx, dw = _lib.rmsnorm_add_bwd(s, s, w, rstd, s, variant=1)
    xh = ref.d(s[-tail:]) * ref.d(rstd[-tail:])[:, None]
    ref.check_gradients(dx[-tail:], None, xh, s[-tail:], s[-tail:], w, rstd[-tail:], 1, False)


@pytest.mark.parametrize("M,N", [(300, 512), (41, 1001), (3, 20000)])
def test_gradient_in_place_of_the_streams(M, N):
    """dx may take the memory of ds."""
    lib = _lib.load()
    x, res, w, dy, ds = inputs(42, M, N)
    _, s, rstd = _lib.rmsnorm_add_fwd(x, res, w, EPS, variant=1)
    want, _ = _lib.rmsnorm_add_bwd(s, dy, w, rstd, ds, need_dw=False, variant=1)
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    assert lib.rmsnorm_add_bwd(p(s), None, p(dy), None, p(ds), None, p(w), p(rstd), p(ds), None, M,
                               N, 1, 0, 1, None, 0, torch.cuda.current_stream().cuda_stream) == 0
    ref.same("dx", ds, want)
