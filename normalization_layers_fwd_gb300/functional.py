"""Autograd wrappers over the C ABI: first-order gradients, like the
``once_differentiable`` backward of the fused-RMSNorm page (DeepSpeed PR 8645
quoted in PR 8664, "Where the kernels run").  Double backward raises.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _lib


def _keep(x, checkpoint, group):
    """What a layer keeps of its input for the backward: x itself, or its 8-bit
    checkpoint (checkpoint: torch.float8_e4m3fn or torch.int8)."""
    return (x,) if checkpoint is None else _lib.act_pack8(x, checkpoint, group)


def _kept(kept, dtype, group):
    """The input again, from what _keep returned."""
    return kept[0] if len(kept) == 1 else _lib.act_unpack8(*kept, dtype, group)


class _DyT(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, alpha, gamma, beta, checkpoint, group):
        ctx.save_for_backward(alpha, gamma, *_keep(x, checkpoint, group))
        ctx.group = group
        return _lib.dyt_fwd(x, alpha, gamma, beta).view(x.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        alpha, gamma, *kept = ctx.saved_tensors
        x = _kept(kept, dy.dtype, ctx.group)
        dx, da, dg, db = _lib.dyt_bwd(x, dy, alpha, gamma, *ctx.needs_input_grad[1:4])
        return dx.view(x.shape), da, dg, db, None, None


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gamma, beta, eps, checkpoint, group):
        y, mean, rstd = _lib.layernorm_fwd(x, gamma, beta, eps)
        ctx.save_for_backward(gamma, mean, rstd, *_keep(x, checkpoint, group))
        ctx.group = group
        ctx.param_dtype = (gamma if gamma is not None else beta).dtype if (
            gamma is not None or beta is not None) else torch.float32
        return y.view(x.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        gamma, mean, rstd, *kept = ctx.saved_tensors
        x = _kept(kept, dy.dtype, ctx.group)
        dx, dg, db = _lib.layernorm_bwd(x, dy, mean, rstd, gamma, ctx.needs_input_grad[1],
                                        ctx.needs_input_grad[2], ctx.param_dtype)
        return dx.view(x.shape), dg, db, None, None, None


class _RMSNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, eps, variant):
        y, rstd = _lib.rmsnorm_fwd(x, w, eps, variant=variant)
        ctx.save_for_backward(x, w, rstd)
        ctx.eps, ctx.variant = eps, variant
        return y.view(x.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w, rstd = ctx.saved_tensors
        dx, dw = _lib.rmsnorm_bwd(x, dy, w, rstd, ctx.eps, ctx.needs_input_grad[1],
                                  variant=ctx.variant)
        return dx.view(x.shape), dw, None, None


class _AddRMSNorm(torch.autograd.Function):
    """y (and, with a residual, the stream s) of the RMSNorm of x + residual."""

    @staticmethod
    def forward(ctx, x, residual, w, eps, variant, checkpoint, group):
        ctx.set_materialize_grads(False)
        ctx.variant, ctx.group, ctx.dtype = variant, group, x.dtype
        if checkpoint is None:
            y, s, rstd = _lib.rmsnorm_add_fwd(x, residual, w, eps, variant=variant)
            ctx.save_for_backward(w, rstd, s)
        else:
            y, s, rstd, c, cscale = _lib.rmsnorm_add_ckpt_fwd(x, residual, w, eps, checkpoint,
                                                              group, variant)
            ctx.save_for_backward(w, rstd, c, cscale)
        return y if residual is None else (y, s)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, ds=None):
        w, rstd, *kept = ctx.saved_tensors
        need_x, need_r, need_w = ctx.needs_input_grad[:3]
        if dy is None:  # y was not used: the norm passes nothing back
            dx, dw = ds, None
        elif len(kept) == 1:
            dx, dw = _lib.rmsnorm_add_bwd(kept[0], dy, w, rstd, ds, need_w, ctx.variant)
        else:
            dx, dw = _lib.rmsnorm_add_ckpt_bwd(*kept, dy, w, rstd, ds, ctx.group, need_w,
                                               ctx.variant)
        if dw is not None:
            dw = dw.view(w.shape)
        return (dx if need_x else None, dx if need_r else None, dw if need_w else None, None, None,
                None, None)


def dyt(x, alpha, gamma, beta, checkpoint=None, group=128):
    """Dynamic Tanh: gamma * tanh(alpha * x) + beta over the last dimension.
    checkpoint (torch.float8_e4m3fn or torch.int8) keeps x for the backward in
    8 bits with a scale per `group` columns (0: per row); then the gradients
    are those at the kept values."""
    return _DyT.apply(x, alpha, gamma, beta, checkpoint, group)


def layer_norm(x, gamma=None, beta=None, eps=1e-5, checkpoint=None, group=128):
    """LayerNorm over the last dimension (biased variance).  checkpoint and
    group as in dyt; the mean and rstd kept are x's own."""
    return _LayerNorm.apply(x, gamma, beta, eps, checkpoint, group)


def rms_norm(x, weight, eps=1e-6, variant=_lib.GBN_RMS_CAST_FIRST, checkpoint=None, group=128):
    """RMSNorm over the last dimension.  variant 0 (default) is the Llama
    expression weight * (x.float() * rsqrt(mean(x^2) + eps)).to(x.dtype);
    1 multiplies by the weight before the cast; 2 is Gemma's (1 + weight)
    before the cast.  checkpoint and group as in dyt; the rstd kept is x's own,
    and the checkpoint is written in the forward's pass."""
    if checkpoint is None:
        return _RMSNorm.apply(x, weight, eps, variant)
    return _AddRMSNorm.apply(x, None, weight, eps, variant, checkpoint, group)


def add_rms_norm(x, residual, weight, eps=1e-6, variant=_lib.GBN_RMS_CAST_FIRST, checkpoint=None,
                 group=128):
    """(y, s): the residual stream s = x + residual (in x's type) and y, the
    RMSNorm of s.  The backward adds the gradient that reaches s from its
    other readers in the same pass; x and residual get the same gradient.
    checkpoint and group as in dyt: s is kept in 8 bits, so the stream itself
    need not live until the backward.  (Without a residual: rms_norm.)"""
    if residual is None:
        raise ValueError("residual is required: rms_norm is the norm without one")
    return _AddRMSNorm.apply(x, residual, weight, eps, variant, checkpoint, group)


def add_rms_norm_quant(x, residual, weight, eps=1e-6, dtype=torch.float8_e4m3fn, group=0,
                       variant=_lib.GBN_RMS_WEIGHT_FIRST):
    """(q, scale, s) for an 8-bit product: y as q * scale (dtype float8_e4m3fn
    or int8, one f32 scale per row, or per 32, 64 or 128 columns) and the
    stream s.  Without a gradient; call it where none is recorded."""
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad
                                       for t in (x, residual, weight)):
        raise RuntimeError("add_rms_norm_quant has no gradient: use add_rms_norm, or call it under "
                           "torch.no_grad()")
    q, scale, s, _ = _lib.rmsnorm_add_quant_fwd(x, residual, weight, eps, dtype, group,
                                                save_rstd=False, variant=variant)
    return q, scale, s
