"""The sequence operators as torch autograd functions.

seq.py takes these where gradients are being recorded and an input requires one; the
calls, their checks and their results are the same.  Gradients are those of the `_grad`
calls; second derivatives are not recorded, and none goes through `final_state`.
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


class GatedScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, native, x, gate, activation, heads, state, final_state, saved):
        ctx.native, ctx.activation = native, activation
        if saved is None:
            saved = native.gated_scan_saved(x)
        y = native.gated_scan(x, gate, activation, heads, state, final_state, saved, None)
        ctx.save_for_backward(x, gate, heads, state, saved)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, gate, heads, state, saved = ctx.saved_tensors
        g = ctx.native.gated_scan_grad(dy.contiguous(), x, gate, ctx.activation, heads, state, saved, None)
        return _wanted(ctx, (None, g["x"], g["gate"], None, None, g.get("state"), None, None))


class LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, native, x, weight, bias, eps, rms, residual, saved):
        ctx.native, ctx.rms = native, rms
        ctx.set_materialize_grads(False)
        if saved is None:
            saved = native.layer_norm_saved(x)
        y = native.layer_norm(x, weight, bias, eps, rms, residual, saved, None)
        ctx.save_for_backward(x if residual is None else y[1], weight, bias, saved)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dsum=None):
        x, weight, bias, saved = ctx.saved_tensors
        if dy is None:  # only the sum was used
            g = {"x": dsum}
        else:
            # sums over tokens only for what asks for them
            need_w, need_b = ctx.needs_input_grad[2:4]
            g = ctx.native.layer_norm_grad(dy.contiguous(), x, weight, bias, ctx.rms, saved,
                                           None if dsum is None else dsum.contiguous(), need_w, need_b)
        parameters = (None if t is None or name not in g else g[name].to(t.dtype)
                      for name, t in (("weight", weight), ("bias", bias)))
        return _wanted(ctx, (None, g["x"], *parameters, None, None, g["x"], None))


class ExpertGather(torch.autograd.Function):
    @staticmethod
    def forward(ctx, native, x, offsets, place):
        ctx.native = native
        ctx.save_for_backward(offsets, place)
        return native.expert_gather(x, offsets, place, None)

    @staticmethod
    @once_differentiable
    def backward(ctx, drows):
        offsets, place = ctx.saved_tensors
        return None, ctx.native.expert_gather_grad(drows.contiguous(), offsets, place, None), None, None


class ExpertCombine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, native, y, offsets, place, weights):
        ctx.native = native
        ctx.save_for_backward(y, offsets, place, weights)
        return native.expert_combine(y, offsets, place, weights, None)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        y, offsets, place, weights = ctx.saved_tensors
        g = ctx.native.expert_combine_grad(dout.contiguous(), y, offsets, place, weights)
        return _wanted(ctx, (None, g["y"], None, None, g.get("weights")))


class Step(torch.autograd.Function):
    """A single-token form: its result can be used, but not differentiated."""

    @staticmethod
    def forward(ctx, name, call, *args):
        ctx.name = name
        return call(*args)

    @staticmethod
    def backward(ctx, dy):
        raise RuntimeError("%s has no gradient: train with %s" % (ctx.name, ctx.name[:-len("_step")]))
