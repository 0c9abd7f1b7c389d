"""The layer as a torch.autograd.Function: moe_forward on the way in, moe_backward on the way back; and its two
ends on their own, ``dispatch`` (moe_permute / moe_permute_backward) and ``combine`` (moe_combine /
moe_combine_backward), for experts of the caller's between them.

Training is the setting of the kieve-moe Features (load-balancing auxiliary loss), the MoEEvolve README
(Architecture) and MoEFFN.forward in moe_stream.py.  ``MoEFunction.apply`` returns the layer output; the
load-balance statistic aux enters the gradient with weight ``aux_coef`` (L = loss(out) + aux_coef * aux), so
the aux value returned by ``moe_layer(..., return_aux=True)`` is for logging and must not be added to the loss
again.  Gradients flow to x, W_r, the routed experts' w13 and w2 and the shared expert's; the routing decision
and the exploration bias take none.  bf16 experts only.  The weight gradients are computed in fp32 and handed
to autograd, which casts them to the parameters' dtype.

Nothing is kept from the forward but its inputs: the backward recomputes the routing and the experts' [g | u].
"""

from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (MoeShape, moe_backward, moe_combine, moe_combine_backward, moe_forward, moe_permute,
               moe_permute_backward)


class MoEFunction(torch.autograd.Function):
    """Inputs: shape (MoeShape), aux_coef (float), x [T, d] bf16, w_router [E, d] fp32, bias [E] fp32 or None,
    w13 [E, 2H, d] bf16, w2 [E, d, H] bf16, w13_sh / w2_sh (or None)."""

    @staticmethod
    def forward(ctx, shape: MoeShape, aux_coef: float, x, w_router, bias, w13, w2, w13_sh, w2_sh):
        r = moe_forward(shape, x, w_router, w13, w2, bias=bias, w13_sh=w13_sh, w2_sh=w2_sh, aux=True)
        ctx.shape, ctx.aux_coef = shape, float(aux_coef)
        ctx.save_for_backward(x, w_router, bias if bias is not None else torch.empty(0), w13, w2,
                              w13_sh if w13_sh is not None else torch.empty(0),
                              w2_sh if w2_sh is not None else torch.empty(0))
        ctx.has = (bias is not None, w13_sh is not None)
        ctx.mark_non_differentiable(r["aux"])
        return r["out"], r["aux"]

    @staticmethod
    def backward(ctx, dout, _daux):
        x, w_router, bias, w13, w2, w13_sh, w2_sh = ctx.saved_tensors
        has_bias, has_sh = ctx.has
        g = moe_backward(ctx.shape, x, w_router, w13, w2, dout.to(torch.bfloat16).contiguous(),
                         bias=bias if has_bias else None, w13_sh=w13_sh if has_sh else None,
                         w2_sh=w2_sh if has_sh else None, aux_coef=ctx.aux_coef)
        return (None, None, g["dx"], g["dw_router"], None, g["dw13"], g["dw2"],
                g["dw13_sh"] if has_sh else None, g["dw2_sh"] if has_sh else None)


def moe_layer(shape: MoeShape, x, w_router, w13, w2, *, bias=None, w13_sh=None, w2_sh=None, aux_coef=0.0,
              return_aux=False):
    """Differentiable routed MoE layer (bf16 experts).  Returns out [T, d] bf16, and aux [1] fp32 (detached)
    when ``return_aux``."""
    out, aux = MoEFunction.apply(shape, aux_coef, x, w_router, bias, w13, w2, w13_sh, w2_sh)
    return (out, aux) if return_aux else out


class DispatchFunction(torch.autograd.Function):
    """Inputs: shape, x [T, d] bf16, topk_idx [T, k] int32.  Outputs: x_perm [R, d] bf16 (differentiable), slot_pos,
    kept, offsets."""

    @staticmethod
    def forward(ctx, shape: MoeShape, x, topk_idx):
        p = moe_permute(shape, x, topk_idx)
        ctx.shape = shape
        ctx.save_for_backward(p["slot_pos"])
        ctx.mark_non_differentiable(p["slot_pos"], p["kept"], p["offsets"])
        return p["x_perm"], p["slot_pos"], p["kept"], p["offsets"]

    @staticmethod
    @once_differentiable
    def backward(ctx, dx_perm, _dslot, _dkept, _doffsets):
        slot_pos, = ctx.saved_tensors
        return None, moe_permute_backward(ctx.shape, dx_perm.contiguous(), slot_pos, dtype=torch.bfloat16), None


def dispatch(shape: MoeShape, x, topk_idx):
    """Differentiable moe_permute: (x_perm [R, d], slot_pos [T, k], kept [E], offsets [E + 1]).  The gradient of a
    token is the sum of its kept rows' gradients; rows that no token fills (zero in x_perm) pass none back."""
    return DispatchFunction.apply(shape, x, topk_idx)


class CombineFunction(torch.autograd.Function):
    """Inputs: shape, y_perm [R, d] bf16, slot_pos, topk_w [T, k] fp32, y_shared [T, d] bf16 or None, kept or None."""

    @staticmethod
    def forward(ctx, shape: MoeShape, y_perm, slot_pos, topk_w, y_shared, kept):
        ctx.shape = shape
        ctx.has_kept = kept is not None and shape.capacity > 0
        ctx.save_for_backward(y_perm, slot_pos, topk_w, kept if ctx.has_kept else torch.empty(0))
        return moe_combine(shape, y_perm, slot_pos, topk_w, y_shared)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        y_perm, slot_pos, topk_w, kept = ctx.saved_tensors
        dout = dout.contiguous()
        need_y, need_w, need_sh = ctx.needs_input_grad[1], ctx.needs_input_grad[3], ctx.needs_input_grad[4]
        g = dict(dy_perm=None, dtopk_w=None)
        if need_y:
            g = moe_combine_backward(ctx.shape, dout, y_perm, slot_pos, topk_w, kept=kept if ctx.has_kept else None,
                                     want_dw=need_w)
        elif need_w:   # frozen rows: no buffer of their size
            g = moe_combine_backward(ctx.shape, dout, y_perm, slot_pos, topk_w, want_dy=False)
        return None, g["dy_perm"], None, g["dtopk_w"], dout if need_sh else None, None


def combine(shape: MoeShape, y_perm, slot_pos, topk_w, y_shared=None, kept=None):
    """Differentiable moe_combine.  Gradients flow to y_perm, topk_w and y_shared; with a capacity give ``kept`` (of
    dispatch), so that the gradient of rows that no token fills is zero."""
    if shape.capacity > 0 and kept is None and y_perm.requires_grad:
        raise ValueError("combine: with a capacity, the gradient of y_perm needs kept")
    dims = dict(y_perm=(shape.R, shape.d), slot_pos=(shape.T, shape.k), topk_w=(shape.T, shape.k),
                y_shared=(shape.T, shape.d))
    for (name, want), t in zip(dims.items(), (y_perm, slot_pos, topk_w, y_shared)):
        if t is not None and tuple(t.shape) != want:   # the gradients' shapes
            raise ValueError(f"combine: {name}: expected shape {want}, got {tuple(t.shape)}")
    return CombineFunction.apply(shape, y_perm, slot_pos, topk_w, y_shared, kept)
