"""Refusals of the residual-stream operators, without a GPU: the C ABI checks
its arguments before it looks for a device."""
import ctypes

import pytest
import torch

from normalization_layers_fwd_gb300 import _lib

OK, EINVAL, EDTYPE, EDEVICE = 0, 1, 2, 5
P = ctypes.c_void_p(64)
ODD = ctypes.c_void_p(65)
E4, I8 = 8, 9


@pytest.fixture(scope="module")
def lib():
    from normalization_layers_fwd_gb300 import build
    build.build()
    return _lib.load()


def fwd(lib, x=P, xl=None, res=P, rl=None, w=P, s=P, y=P, rstd=None, M=4, N=8, eps=1e-6, xt=1,
        wt=1, variant=0):
    return lib.rmsnorm_add_fwd(x, xl, res, rl, w, s, y, rstd, M, N, eps, xt, wt, variant, None)


def quant(lib, x=P, res=P, w=P, s=P, q=P, scale=P, rstd=None, M=4, N=8, group=0, eps=1e-6, xt=1,
          wt=1, qt=E4, variant=1):
    return lib.rmsnorm_add_quant_fwd(x, None, res, None, w, s, q, scale, rstd, M, N, group, eps,
                                     xt, wt, qt, variant, None)


def ckpt_fwd(lib, x=P, res=P, w=P, s=P, y=P, rstd=P, c=P, cscale=P, M=4, N=8, group=32, ct=I8):
    return lib.rmsnorm_add_ckpt_fwd(x, None, res, None, w, s, y, rstd, c, cscale, M, N, group,
                                    1e-6, 1, 1, ct, 0, None)


def bwd(lib, s=P, sl=None, dy=P, dyl=None, ds=P, dsl=None, w=P, rstd=P, dx=P, dw=None, M=4, N=8,
        xt=1, wt=1, variant=0, ws=None, n=0):
    return lib.rmsnorm_add_bwd(s, sl, dy, dyl, ds, dsl, w, rstd, dx, dw, M, N, xt, wt, variant, ws,
                               n, None)


def ckpt_bwd(lib, c=P, cscale=P, dy=P, ds=P, w=P, rstd=P, dx=P, dw=None, M=4, N=8, group=64,
             ct=E4, ws=None, n=0):
    return lib.rmsnorm_add_ckpt_bwd(c, cscale, dy, None, ds, None, w, rstd, dx, dw, M, N, group, 1,
                                    1, ct, 0, ws, n, None)


def pack(lib, x=P, c=P, cscale=P, M=4, N=8, group=32, xt=1, ct=E4, xl=None):
    return lib.act_pack8(x, xl, c, cscale, M, N, group, xt, ct, None)


def unpack(lib, c=P, cscale=P, x=P, M=4, N=8, group=32, xt=1, ct=E4):
    return lib.act_unpack8(c, cscale, x, M, N, group, xt, ct, None)


CALLS = (fwd, quant, ckpt_fwd, bwd, ckpt_bwd, pack, unpack)


@pytest.mark.parametrize("call", CALLS)
def test_bad_shapes(lib, call):
    for kw in (dict(M=-1), dict(N=0), dict(N=-8), dict(N=1 << 31), dict(M=1 << 60)):
        assert call(lib, **kw) == EINVAL, kw


@pytest.mark.parametrize("call", CALLS)
def test_valid_calls_get_as_far_as_the_device(lib, call):
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    assert call(lib) == EDEVICE


@pytest.mark.parametrize("call,names", [
    (fwd, ("x", "w", "y")), (quant, ("x", "w", "q", "scale")),
    (ckpt_fwd, ("x", "w", "y", "c", "cscale")), (bwd, ("s", "dy", "w", "rstd", "dx")),
    (ckpt_bwd, ("c", "cscale", "dy", "w", "rstd", "dx")), (pack, ("x", "c", "cscale")),
    (unpack, ("c", "cscale", "x"))])
def test_required_pointers(lib, call, names):
    for n in names:
        assert call(lib, **{n: None}) == EINVAL, n


@pytest.mark.parametrize("call,names", [
    (fwd, ("x", "res", "w", "s", "y", "rstd")), (quant, ("x", "res", "w", "s", "scale", "rstd")),
    (ckpt_fwd, ("x", "res", "s", "y", "rstd", "cscale")),
    (bwd, ("s", "dy", "ds", "w", "rstd", "dx", "dw")),
    (ckpt_bwd, ("cscale", "dy", "ds", "w", "rstd", "dx", "dw")), (pack, ("x", "cscale")),
    (unpack, ("cscale", "x"))])
def test_misaligned_pointers(lib, call, names):
    for n in names:
        assert call(lib, **{n: ODD}) == EINVAL, n


def test_eight_bit_pointers_take_any_alignment(lib):
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    assert quant(lib, q=ODD) == ckpt_fwd(lib, c=ODD) == pack(lib, c=ODD) == EDEVICE
    assert unpack(lib, c=ODD) == ckpt_bwd(lib, c=ODD) == EDEVICE


def test_stream_output_needs_a_residual(lib):
    assert fwd(lib, res=None) == EINVAL
    assert quant(lib, res=None) == EINVAL
    if not torch.cuda.is_available():
        assert fwd(lib, res=None, s=None) == EDEVICE
        assert fwd(lib, s=None) == EDEVICE


@pytest.mark.parametrize("call", [quant, ckpt_fwd, ckpt_bwd, pack, unpack])
def test_groups_and_eight_bit_types(lib, call):
    t = {quant: "qt"}.get(call, "ct")
    for g in (-1, 1, 16, 33, 256, 1 << 40):
        assert call(lib, group=g) == EINVAL
    for code in (0, 1, 2, 3, 7, 10, -1):
        assert call(lib, **{t: code}) == EDTYPE


def test_types_and_expressions(lib):
    for call in (fwd, quant, bwd):
        assert call(lib, xt=3) == EDTYPE
        assert call(lib, wt=8) == EDTYPE
        assert call(lib, variant=3) == EINVAL
        assert call(lib, variant=-1) == EINVAL
    # expression 0 rounds to the activations' type: no weight of the other 16-bit type
    assert fwd(lib, xt=1, wt=2, variant=0) == EDTYPE
    assert bwd(lib, xt=2, wt=1, variant=0) == EDTYPE
    assert pack(lib, xt=8) == EDTYPE and unpack(lib, xt=-1) == EDTYPE
    for eps in (float("nan"), float("inf"), -1e-6):
        assert fwd(lib, eps=eps) == EINVAL and quant(lib, eps=eps) == EINVAL


def test_layouts(lib):
    bad = _lib.gbn_rows(0, 8, 1, 0, 0)
    far = _lib.gbn_rows(4, 1 << 61, 1, 0, 0)
    for lay in (bad, far):
        r = ctypes.byref(lay)
        assert fwd(lib, xl=r) == fwd(lib, rl=r) == bwd(lib, sl=r) == EINVAL
        assert bwd(lib, dyl=r) == bwd(lib, dsl=r) == pack(lib, xl=r) == EINVAL


def test_workspace(lib):
    assert bwd(lib, dw=P, ws=ctypes.c_void_p(66), n=1 << 20) == EINVAL
    size_max = ctypes.c_size_t(-1).value
    assert lib.gbn_bwd_workspace_bytes(3, 0, 8, 1, 1, 0) == 0
    assert lib.gbn_bwd_workspace_bytes(3, -1, 8, 1, 1, 0) == size_max
    assert lib.gbn_bwd_workspace_bytes(4, 4, 8, 1, 1, 0) == size_max


def test_empty_forwards_need_no_device(lib):
    assert lib.rmsnorm_add_fwd(None, None, None, None, P, None, None, None, 0, 8, 1e-6, 1, 1, 0,
                               None) == OK
    assert lib.act_pack8(None, None, None, None, 0, 8, 32, 1, E4, None) == OK
    assert lib.act_unpack8(None, None, None, 0, 8, 32, 1, E4, None) == OK


def test_binding_refuses_before_the_library(lib):
    x, w = torch.zeros(4, 8), torch.ones(8)
    for f in (lambda: _lib.rmsnorm_add_fwd(x, x, w), lambda: _lib.act_pack8(x),
              lambda: _lib.rmsnorm_add_quant_fwd(x, x, w),
              lambda: _lib.rmsnorm_add_ckpt_fwd(x, None, w),
              lambda: _lib.rmsnorm_add_bwd(x, x, w, torch.ones(4)),
              lambda: _lib.act_unpack8(torch.zeros(4, 8, dtype=torch.int8), torch.ones(4, 1))):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        _lib.act_pack8(x, torch.uint8)
    with pytest.raises(TypeError):
        _lib.rmsnorm_add_quant_fwd(x, x, w, dtype=torch.float8_e5m2)


def test_wrappers_refuse():
    from normalization_layers_fwd_gb300 import functional as F
    x, w = torch.zeros(4, 64), torch.ones(64)
    with pytest.raises(ValueError, match="residual"):
        F.add_rms_norm(x, None, w)
    with pytest.raises(RuntimeError, match="no gradient"):
        F.add_rms_norm_quant(x.requires_grad_(), x, w)
    with pytest.raises(ValueError):
        F.rms_norm(x, w, checkpoint=torch.int8)
