"""Sequence-model operators: token embedding, short causal convolution, selective
state space scan, gated recurrence, norm, and the way of tokens to their experts and
back (binding over ``include/sc_seq.h``).

The functions take torch CUDA tensors and run on the current torch stream (or
``stream``); they check shapes and types (ValueError), allocate what they return
(on that stream), and leave every step of the computation to the library's
kernels.  Definitions, layouts and limits: the header.

embed, causal_conv, selective_scan, gated_scan, layer_norm, expert_gather and
expert_combine are differentiable: where torch records gradients and an input requires
one, their results carry it (seq_autograd.py), by the `_grad` functions below, which may
also be called by themselves.  `out` cannot be given then, and nothing goes back through
`final_state`.  The `_step` forms have no gradient; asking for one raises.  Forward-mode
derivatives are not recorded either: a tensor with a tangent is refused
(NotImplementedError).

    ids, weight                 y = embed(ids, weight, scale)
                                dweight = embed_grad(ids, dy, vocab, scale)
    x (batch, length, channels) y = causal_conv(x, weight, bias)
                                grads = causal_conv_grad(dy, x, weight, bias)
                                y = causal_conv_step(x1, state, weight, bias)
    x, dt, A, B, C              y = selective_scan(x, dt, A, B, C, D, z, dt_bias)
                                grads = selective_scan_grad(dy, x, ..., saved=saved)
                                y = selective_scan_step(x1, dt1, A, B1, C1, state)
    x, gate                     y = gated_scan(x, gate)
                                grads = gated_scan_grad(dy, x, gate, saved=saved)
                                y = gated_scan_step(x1, gate1, state)
    x (..., channels), residual y, sum = layer_norm(x, weight, bias, residual=residual)
                                grads = layer_norm_grad(dy, sum, weight, bias, saved=saved, dsum=dsum)
    experts (tokens, choices)   order = expert_sort(experts, n_experts)
    x (tokens, dim)             rows = expert_gather(x, order)
                                y = expert_combine(rows, order, weights)
"""
from __future__ import annotations

import ctypes
from typing import Any, NamedTuple

SC_F16, SC_BF16 = 8, 9
SC_CONV_MAX_WIDTH, SC_SSM_MAX_STATES, SC_SSM_SAVE = 8, 64, 16
SC_GATED_SAVE, SC_EXPERT_MAX = 16, 1024

_P, _I64, _I32, _INT, _SZ, _F = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int, ctypes.c_size_t,
                                ctypes.c_float)


class ConvDesc(ctypes.Structure):
    """sc_conv_desc."""
    _fields_ = [("dtype", _I32), ("width", _I32), ("silu", _I32), ("reserved", _I32), ("batch", _I64),
                ("length", _I64), ("channels", _I64), ("x", _P), ("x_batch", _I64), ("x_token", _I64),
                ("weight", _P), ("bias", _P), ("heads", _P), ("state", _P)]


class SsmDesc(ctypes.Structure):
    """sc_ssm_desc."""
    _fields_ = [("dtype", _I32), ("softplus", _I32), ("batch", _I64), ("length", _I64), ("channels", _I64),
                ("states", _I64), ("groups", _I64), ("x", _P), ("dt", _P), ("x_batch", _I64), ("x_token", _I64),
                ("dt_batch", _I64), ("dt_token", _I64), ("A", _P), ("B", _P), ("C", _P), ("B_batch", _I64),
                ("B_token", _I64), ("B_group", _I64), ("C_batch", _I64), ("C_token", _I64), ("C_group", _I64),
                ("D", _P), ("z", _P), ("z_batch", _I64), ("z_token", _I64), ("dt_bias", _P), ("heads", _P),
                ("state", _P)]


class SsmGrads(ctypes.Structure):
    """sc_ssm_grads."""
    _fields_ = [("dy", _P), ("dy_batch", _I64), ("dy_token", _I64), ("saved", _P), ("dfinal", _P), ("dx", _P),
                ("ddt", _P), ("dz", _P), ("dB", _P), ("dC", _P), ("dA", _P), ("dD", _P), ("ddt_bias", _P),
                ("dstate", _P)]


class GatedDesc(ctypes.Structure):
    """sc_gated_desc."""
    _fields_ = [("dtype", _I32), ("sigmoid", _I32), ("batch", _I64), ("length", _I64), ("channels", _I64), ("x", _P),
                ("gate", _P), ("x_batch", _I64), ("x_token", _I64), ("gate_batch", _I64), ("gate_token", _I64),
                ("heads", _P), ("state", _P)]


class NormDesc(ctypes.Structure):
    """sc_norm_desc."""
    _fields_ = [("dtype", _I32), ("wtype", _I32), ("rms", _I32), ("eps", _F), ("batch", _I64), ("length", _I64),
                ("channels", _I64), ("x", _P), ("x_batch", _I64), ("x_token", _I64), ("residual", _P),
                ("residual_batch", _I64), ("residual_token", _I64), ("weight", _P), ("bias", _P)]


class ExpertDesc(ctypes.Structure):
    """sc_expert_desc."""
    _fields_ = [("dtype", _I32), ("wtype", _I32), ("tokens", _I64), ("choices", _I64), ("dim", _I64),
                ("experts", _I64), ("place", _P), ("offsets", _P), ("weights", _P)]


_CONV, _SSM, _GRADS = ctypes.POINTER(ConvDesc), ctypes.POINTER(SsmDesc), ctypes.POINTER(SsmGrads)
_GATED, _NORM, _EXPERT = ctypes.POINTER(GatedDesc), ctypes.POINTER(NormDesc), ctypes.POINTER(ExpertDesc)

SIGNATURES = {
    "sc_embed": ([_P, _INT, _I64, _INT, _P, _I64, _I64, _I64, _F, _P, _I64, _P], _INT),
    "sc_embed_grad": ([_P, _INT, _I64, _INT, _P, _I64, _I64, _I64, _F, _INT, _P, _I64, _INT, _P], _INT),
    "sc_embed_grad_workspace_bytes": ([_I64, _I64, _I64], _SZ),
    "sc_causal_conv": ([_CONV, _P, _I64, _I64, _P, _P], _INT),
    "sc_causal_conv_grad": ([_CONV, _P, _I64, _I64, _P, _I64, _I64, _P, _P, _P, _P], _INT),
    "sc_causal_conv_grad_workspace_bytes": ([_I64, _I64, _I64, _INT], _SZ),
    "sc_causal_conv_step": ([_CONV, _P, _I64, _P, _P, _I64, _P], _INT),
    "sc_selective_scan": ([_SSM, _P, _I64, _I64, _P, _P, _P], _INT),
    "sc_selective_scan_saved_bytes": ([_I64, _I64, _I64, _I64], _SZ),
    "sc_selective_scan_workspace_bytes": ([_I64, _I64, _I64, _I64, _I64], _SZ),
    "sc_selective_scan_grad": ([_SSM, _GRADS, _P], _INT),
    "sc_selective_scan_grad_workspace_bytes": ([_I64, _I64, _I64, _I64, _I64], _SZ),
    "sc_selective_scan_step": ([_SSM, _P, _I64, _P, _P, _I64, _P], _INT),
    "sc_gated_scan": ([_GATED, _P, _I64, _I64, _P, _P, _P], _INT),
    "sc_gated_scan_saved_bytes": ([_I64, _I64, _I64], _SZ),
    "sc_gated_scan_grad": ([_GATED, _P, _I64, _I64, _P, _P, _P, _P, _P, _P], _INT),
    "sc_gated_scan_step": ([_GATED, _P, _I64, _P, _P, _I64, _P], _INT),
    "sc_layer_norm": ([_NORM, _P, _I64, _I64, _P, _I64, _I64, _P, _P], _INT),
    "sc_layer_norm_grad": ([_NORM, _P, _I64, _I64, _P, _I64, _I64, _P, _P, _P, _P, _P], _INT),
    "sc_layer_norm_grad_workspace_bytes": ([_I64, _I64, _I64, _INT], _SZ),
    "sc_expert_sort": ([_P, _INT, _I64, _I64, _P, _P, _P, _P], _INT),
    "sc_expert_gather": ([_EXPERT, _P, _I64, _P, _I64, _P], _INT),
    "sc_expert_gather_grad": ([_EXPERT, _P, _I64, _P, _I64, _P], _INT),
    "sc_expert_combine": ([_EXPERT, _P, _I64, _P, _I64, _P], _INT),
    "sc_expert_combine_grad": ([_EXPERT, _P, _I64, _P, _I64, _P, _I64, _P, _P], _INT),
}


# ------------------------------------------------------------ tensor layer
# The functions are compiled (csrc/sc_bind.cpp); here are their arguments and
# what they mean.  Those of the block's operators return None where a gradient is to be
# recorded, and the call goes through its autograd function instead.
_bind = None


def _native():
    global _bind
    if _bind is None:
        from . import load
        load()
        import torch  # noqa: F401  (its libraries, before the binding's)
        try:
            from . import _seqbind
        except ImportError as e:
            raise RuntimeError("the binding of the sequence operators is not built; run "
                               "`python -m stream_compaction_gb300.build`") from e
        _bind = _seqbind
    return _bind


def _call(name, stream, *args):
    if stream is None:
        return getattr(_bind or _native(), name)(*args)
    import torch
    with torch.cuda.stream(stream):  # what the call allocates belongs to the stream that it runs on
        return getattr(_native(), name)(*args)


def _requires_grad(*tensors) -> bool:
    for t in tensors:
        if t is not None and getattr(t, "requires_grad", False):
            import torch
            return torch.is_grad_enabled()
    return False


def _record(function, stream, out, *args):
    """The call through an autograd function; `out` has no place in it."""
    if out is not None:
        raise ValueError("out cannot be given where an input requires a gradient")
    from . import seq_autograd
    native, apply = _native(), getattr(seq_autograd, function).apply
    if stream is None:
        return apply(native, *args)
    import torch
    with torch.cuda.stream(stream):  # the gradient runs there, too
        return apply(native, *args)


def _step(name, stream, inputs, *args):
    if not _requires_grad(*inputs):
        return _call(name, stream, *args)
    from . import seq_autograd
    return seq_autograd.Step.apply(name, lambda *a: _call(name, stream, *a), *args)


def embed(ids, weight, scale: float = 1.0, out=None, stream=None):
    """scale * weight[ids]: ids (int32 or int64) of any shape, weight (vocab, dim);
    a row of zeros where an id is outside [0, vocab)."""
    if _requires_grad(weight):
        return _record("Embed", stream, out, ids, weight, scale)
    return _call("embed", stream, ids, weight, scale, out)


def embed_grad(ids, dout, vocab: int, scale: float = 1.0, out=None, accumulate: bool = False, stream=None):
    """Gradient of embed by its weight: (vocab, dim), of dout's type unless `out` is
    given (dout's type or float32); accumulate: added to what `out` holds."""
    return _call("embed_grad", stream, ids, dout, vocab, scale, out, accumulate)


def causal_conv(x, weight, bias=None, activation="silu", heads=None, state=None, final_state=None, out=None,
                stream=None):
    """Causal convolution of x (batch, length, channels) with weight (channels,
    width), one filter per channel; activation "silu" or None.  heads: one
    uint8/bool flag per token, nonzero where a segment starts.  state: the width - 1
    inputs before x, oldest first (batch, width - 1, channels); final_state:
    receives those after x."""
    if _requires_grad(x, weight, bias, state):
        return _record("CausalConv", stream, out, x, weight, bias, activation, heads, state, final_state)
    return _call("causal_conv", stream, x, weight, bias, activation, heads, state, final_state, out)


def causal_conv_grad(dy, x, weight, bias=None, activation="silu", heads=None, state=None, stream=None):
    """Gradients of causal_conv: a dict with x (x's type), weight and bias (float32)
    and, where `state` is given, state (x's type)."""
    return _call("causal_conv_grad", stream, dy, x, weight, bias, activation, heads, state)


def causal_conv_step(x, state, weight, bias=None, activation="silu", slots=None, out=None, stream=None):
    """One token for each row of x (batch, channels); state (rows, width - 1,
    channels) is moved on in place.  slots (int32): the state row of each x row,
    no row twice; outside [0, rows): the x row sits out, its y is 0."""
    return _step("causal_conv_step", stream, (x, weight, bias, state), x, state, weight, bias, activation, slots, out)


def selective_scan_saved(x, A, stream=None):
    """The buffer that a selective_scan of x with A fills for selective_scan_grad."""
    return _call("selective_scan_saved", stream, x, A)


def selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus: bool = True, heads=None, state=None,
                   final_state=None, saved=None, out=None, stream=None):
    """Selective state space scan of x (batch, length, channels): dt like x, A
    (channels, states) float32, B and C (batch, length, groups, states), D and
    dt_bias (channels) float32, z like x.  heads as in causal_conv; state /
    final_state: (batch, channels, states) float32.  saved: from
    selective_scan_saved, for selective_scan_grad."""
    if _requires_grad(x, dt, A, B, C, D, z, dt_bias, state):
        return _record("SelectiveScan", stream, out, x, dt, A, B, C, D, z, dt_bias, softplus, heads, state, final_state,
                       saved)
    return _call("selective_scan", stream, x, dt, A, B, C, D, z, dt_bias, softplus, heads, state, final_state, saved,
                 out)


def selective_scan_grad(dy, x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus: bool = True, heads=None,
                        state=None, saved=None, dfinal_state=None, stream=None):
    """Gradients of selective_scan, given what it saved: a dict with x, dt, B, C
    (their types), A, and those of D, z, dt_bias and state that were given."""
    return _call("selective_scan_grad", stream, dy, x, dt, A, B, C, D, z, dt_bias, softplus, heads, state, saved,
                 dfinal_state)


def selective_scan_step(x, dt, A, B, C, state, D=None, z=None, dt_bias=None, softplus: bool = True, slots=None,
                        out=None, stream=None):
    """One token for each row of x (batch, channels), B and C (batch, groups,
    states); state (rows, channels, states) float32 is moved on in place.  slots
    as in causal_conv_step."""
    return _step("selective_scan_step", stream, (x, dt, A, B, C, D, z, dt_bias, state), x, dt, A, B, C, state, D, z,
                 dt_bias, softplus, slots, out)


def gated_scan_saved(x, stream=None):
    """The buffer that a gated_scan of x fills for gated_scan_grad."""
    return _call("gated_scan_saved", stream, x)


def gated_scan(x, gate, activation="sigmoid", heads=None, state=None, final_state=None, saved=None, out=None,
               stream=None):
    """Gated recurrence of x (batch, length, channels), gate like x: h = f * h + (1 - f) * x
    with f = sigmoid(gate), or with activation None h = gate * h + x (gates of any size).
    heads as in causal_conv; state / final_state: (batch, channels) float32.  saved: from
    gated_scan_saved, for gated_scan_grad."""
    y = _call("gated_scan", stream, x, gate, activation, heads, state, final_state, saved, out)
    if y is None:
        return _record("GatedScan", stream, out, x, gate, activation, heads, state, final_state, saved)
    return y


def gated_scan_grad(dy, x, gate, activation="sigmoid", heads=None, state=None, saved=None, dfinal_state=None,
                    stream=None):
    """Gradients of gated_scan, given what it saved: a dict with x and gate (their type)
    and, where `state` is given, state (float32)."""
    return _call("gated_scan_grad", stream, dy, x, gate, activation, heads, state, saved, dfinal_state)


def gated_scan_step(x, gate, state, activation="sigmoid", slots=None, out=None, stream=None):
    """One token for each row of x (batch, channels); state (rows, channels) float32 is
    moved on in place.  slots as in causal_conv_step."""
    y = _call("gated_scan_step", stream, x, gate, state, activation, slots, out)
    if y is None:
        return _step("gated_scan_step", stream, (x, gate, state), x, gate, state, activation, slots, out)
    return y


def layer_norm_saved(x, stream=None):
    """The buffer that a layer_norm of x fills for layer_norm_grad: a row's mean and
    1 / deviation."""
    return _call("layer_norm_saved", stream, x)


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, rms: bool = False, residual=None, saved=None, out=None,
               stream=None):
    """The norm of x (..., channels) over its channels, times weight, plus bias (each
    (channels), of x's type or float32); rms: without the mean.  residual (like x): the
    norm of x + residual, and the result is the pair (y, x + residual), the sum rounded
    to x's type.  saved: from layer_norm_saved, for layer_norm_grad."""
    y = _call("layer_norm", stream, x, weight, bias, eps, rms, residual, saved, out)
    if y is None:
        return _record("LayerNorm", stream, out, x, weight, bias, eps, rms, residual, saved)
    return y


def layer_norm_grad(dy, x, weight=None, bias=None, rms: bool = False, saved=None, dsum=None, stream=None):
    """Gradients of layer_norm at x (the sum, where there was a residual), given what it
    saved: a dict with x (x's type; dsum, what reaches the sum by itself, is added to
    it, and it is the residual's gradient too), and weight and bias (float32) where they
    are given."""
    return _call("layer_norm_grad", stream, dy, x, weight, bias, rms, saved, dsum, True, True)


class ExpertOrder(NamedTuple):
    """What expert_sort returns.  The rows of expert e are offsets[e] to offsets[e + 1]
    (int64, n_experts + 1); order[row] is the entry of a row, token * choices + choice,
    and place[token, choice] the row of an entry (both int32).  Entries of no expert
    are behind offsets[n_experts]."""
    offsets: Any
    order: Any
    place: Any


def expert_sort(experts, n_experts: int, stream=None):
    """The entries of experts (tokens, choices; int32 or int64) in the order of their
    experts, stable; ids outside [0, n_experts) have no expert and come last.
    n_experts: 1 to 1024."""
    return ExpertOrder(*_call("expert_sort", stream, experts, n_experts))


def expert_gather(x, order, out=None, stream=None):
    """A row of x (tokens, dim) for each entry, in the order of the experts (tokens *
    choices, dim); zeros for entries of no expert."""
    y = _call("expert_gather", stream, x, order.offsets, order.place, out)
    if y is None:
        return _record("ExpertGather", stream, out, x, order.offsets, order.place)
    return y


def expert_gather_grad(drows, order, out=None, stream=None):
    """Gradient of expert_gather by x: the sum of a token's rows of drows."""
    return _call("expert_gather_grad", stream, drows, order.offsets, order.place, out)


def expert_combine(y, order, weights=None, out=None, stream=None):
    """The way back: the sum of a token's rows of y (tokens * choices, dim, in the order
    of the experts), times weights (tokens, choices; of y's type or float32) where they
    are given; entries of no expert add nothing."""
    z = _call("expert_combine", stream, y, order.offsets, order.place, weights, out)
    if z is None:
        return _record("ExpertCombine", stream, out, y, order.offsets, order.place, weights)
    return z


def expert_combine_grad(dout, y, order, weights=None, stream=None):
    """Gradients of expert_combine: a dict with y (y's type, zeros for entries of no
    expert) and, where they are given, weights (their type)."""
    return _call("expert_combine_grad", stream, dout, y, order.offsets, order.place, weights)
