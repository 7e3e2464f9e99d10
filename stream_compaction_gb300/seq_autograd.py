"""The sequence operators as torch autograd functions.

seq.py takes these where gradients are being recorded and an input requires one; the
calls, their checks and their results are the same.  Gradients are those of embed_grad,
causal_conv_grad and selective_scan_grad; second derivatives are not recorded, and none
goes through `final_state`.
"""
import torch
from torch.autograd.function import once_differentiable


def _wanted(ctx, grads):
    return tuple(g if need else None for g, need in zip(grads, ctx.needs_input_grad))


class Embed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, native, ids, weight, scale):
        ctx.native, ctx.vocab, ctx.scale = native, weight.shape[0], scale
        ctx.save_for_backward(ids)
        return native.embed(ids, weight, scale, None)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        (ids,) = ctx.saved_tensors
        return None, None, ctx.native.embed_grad(ids, dy.contiguous(), ctx.vocab, ctx.scale, None, False), None


class CausalConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, native, x, weight, bias, activation, heads, state, final_state):
        ctx.native, ctx.activation = native, activation
        y = native.causal_conv(x, weight, bias, activation, heads, state, final_state, None)
        ctx.save_for_backward(x, weight, bias, heads, state)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, bias, heads, state = ctx.saved_tensors
        g = ctx.native.causal_conv_grad(dy.contiguous(), x, weight, bias, ctx.activation, heads, state)
        return _wanted(ctx, (None, g["x"], g["weight"].to(weight.dtype), None if bias is None else g["bias"].to(bias.dtype),
                             None, None, g.get("state"), None))


class SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, native, x, dt, A, B, C, D, z, dt_bias, softplus, heads, state, final_state, saved):
        ctx.native, ctx.softplus = native, softplus
        if saved is None:
            saved = native.selective_scan_saved(x, A)
        y = native.selective_scan(x, dt, A, B, C, D, z, dt_bias, softplus, heads, state, final_state, saved, None)
        ctx.save_for_backward(x, dt, A, B, C, D, z, dt_bias, heads, state, saved)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, dt, A, B, C, D, z, dt_bias, heads, state, saved = ctx.saved_tensors
        g = ctx.native.selective_scan_grad(dy.contiguous(), x, dt, A, B, C, D, z, dt_bias, ctx.softplus, heads, state,
                                           saved, None)
        return _wanted(ctx, (None, g["x"], g["dt"], g["A"], g["B"], g["C"], g.get("D"), g.get("z"), g.get("dt_bias"),
                             None, None, g.get("state"), None, None))


class Step(torch.autograd.Function):
    """A single-token form: its result can be used, but not differentiated."""

    @staticmethod
    def forward(ctx, name, call, *args):
        ctx.name = name
        return call(*args)

    @staticmethod
    def backward(ctx, dy):
        raise RuntimeError("%s has no gradient: train with %s" % (ctx.name, ctx.name[:-len("_step")]))
