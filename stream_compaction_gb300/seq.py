"""Sequence-model operators: token embedding, short causal convolution and
selective state space scan (binding over ``include/sc_seq.h``).

The functions take torch CUDA tensors and run on the current torch stream (or
``stream``); they check shapes and types, allocate what they return (on that
stream), and leave every step of the computation to the library's kernels.
Definitions, layouts and limits: the header.

    ids, weight                 y = embed(ids, weight, scale)
                                dweight = embed_grad(ids, dy, vocab, scale)
    x (batch, length, channels) y = causal_conv(x, weight, bias)
                                grads = causal_conv_grad(dy, x, weight, bias)
                                y = causal_conv_step(x1, state, weight, bias)
    x, dt, A, B, C              y = selective_scan(x, dt, A, B, C, D, z, dt_bias)
                                grads = selective_scan_grad(dy, x, ..., saved=saved)
                                y = selective_scan_step(x1, dt1, A, B1, C1, state)
"""
from __future__ import annotations

import contextlib
import ctypes

SC_F16, SC_BF16 = 8, 9
SC_CONV_MAX_WIDTH, SC_SSM_MAX_STATES, SC_SSM_SAVE = 8, 64, 16

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


_CONV, _SSM, _GRADS = ctypes.POINTER(ConvDesc), ctypes.POINTER(SsmDesc), ctypes.POINTER(SsmGrads)

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
}


# ------------------------------------------------------------------ checks
_CODES = None


def _code(t, what: str) -> int:
    global _CODES
    if _CODES is None:
        import torch
        _CODES = {torch.float32: 2, torch.float16: SC_F16, torch.bfloat16: SC_BF16}
    code = _CODES.get(t.dtype)
    if code is None:
        raise ValueError("%s must be float32, float16 or bfloat16, got %s" % (what, t.dtype))
    return code


def _need(ok: bool, message: str) -> None:
    if not ok:
        raise ValueError(message)


def _like(t, what: str, shape, dtype, device):
    """A tensor of this shape and type on the device whose last dimension is contiguous."""
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (what, tuple(shape), tuple(t.shape)))
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (what, dtype, t.dtype))
    if t.device != device:
        raise ValueError("%s must be on %s, got %s" % (what, device, t.device))
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError("%s: elements of the last dimension must be contiguous" % what)
    return t


def _whole(t, what: str, shape, dtype, device):
    """The same, contiguous throughout; the pointer (None: 0)."""
    if t is None:
        return 0
    _like(t, what, shape, dtype, device)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % what)
    return t.data_ptr()


def _cuda(t, what: str) -> None:
    import torch
    if not t.is_cuda:
        raise ValueError("%s: expected a CUDA tensor" % what)
    if t.device.index != torch.cuda.current_device():
        raise ValueError("%s must be on the current CUDA device" % what)


def _heads(heads, shape, device) -> int:
    import torch
    if heads is None:
        return 0
    if heads.dtype not in (torch.uint8, torch.bool, torch.int8):
        raise ValueError("heads must be a uint8/bool tensor with one flag per token")
    return _whole(heads, "heads", shape, heads.dtype, device)


@contextlib.contextmanager
def _allocating_on(stream):
    """What a call allocates belongs to the stream that the call runs on."""
    import torch
    with torch.cuda.stream(stream):
        yield


def _on(stream):
    return contextlib.nullcontext() if stream is None else _allocating_on(stream)


def _lib():
    from . import load
    return load()


def _stream(stream) -> int:
    import torch
    return int((torch.cuda.current_stream() if stream is None else stream).cuda_stream)


def _check(status: int, where: str) -> None:
    if status:
        from . import ScanError
        raise ScanError(status, where)


# --------------------------------------------------------------- embedding
def _ids(ids):
    import torch
    _cuda(ids, "ids")
    _need(ids.dtype in (torch.int32, torch.int64), "ids must be int32 or int64")
    _need(ids.is_contiguous(), "ids must be contiguous")
    return int(ids.dtype == torch.int64)


def embed(ids, weight, scale: float = 1.0, out=None, stream=None):
    """scale * weight[ids]: ids of any shape, weight (vocab, dim); a row of zeros
    where an id is outside [0, vocab)."""
    import torch
    ids64 = _ids(ids)
    code = _code(weight, "weight")
    _need(weight.dim() == 2, "weight must have shape (vocab, dim)")
    vocab, dim = weight.shape
    _like(weight, "weight", weight.shape, weight.dtype, ids.device)
    shape = ids.shape + (dim,)
    if out is None:
        with _on(stream):
            out = torch.empty(shape, dtype=weight.dtype, device=ids.device)
    else:
        _whole(out, "out", shape, weight.dtype, ids.device)
    _check(_lib().sc_embed(ids.data_ptr(), ids64, ids.numel(), code, weight.data_ptr(), vocab, dim,
                           max(weight.stride(0), dim) if vocab < 2 else weight.stride(0), scale, out.data_ptr(), dim,
                           _stream(stream)), "sc_embed")
    return out


def embed_grad(ids, dout, vocab: int, scale: float = 1.0, out=None, accumulate: bool = False, stream=None):
    """Gradient of embed by its weight: (vocab, dim), of dout's type unless `out` is
    given (dout's type or float32); accumulate: added to what `out` holds."""
    import torch
    ids64 = _ids(ids)
    code = _code(dout, "dout")
    _need(dout.dim() >= 1 and dout.shape[:-1] == ids.shape, "dout must have the shape of ids and one dimension more")
    _need(vocab >= 0, "vocab must not be negative")
    _need(out is not None or not accumulate, "accumulate needs `out`")
    dim = dout.shape[-1]
    _like(dout, "dout", dout.shape, dout.dtype, ids.device)
    rows = dout.reshape(-1, dim) if dout.is_contiguous() else dout
    _need(rows.dim() == 2, "dout must be contiguous, or a matrix of rows")
    shape = torch.Size((vocab, dim))
    if out is None:
        with _on(stream):
            out = torch.empty(shape, dtype=dout.dtype, device=ids.device)
    else:
        _need(out.dtype in (dout.dtype, torch.float32), "out must be of dout's type or float32")
        _like(out, "out", shape, out.dtype, ids.device)
    ldd = rows.stride(0) if rows.shape[0] > 1 else dim
    ldw = out.stride(0) if vocab > 1 else dim
    _check(_lib().sc_embed_grad(ids.data_ptr(), ids64, ids.numel(), code, rows.data_ptr(), ldd, vocab, dim, scale,
                                _code(out, "out"), out.data_ptr(), ldw, int(accumulate), _stream(stream)),
           "sc_embed_grad")
    return out


# ------------------------------------------------------------- convolution
_ACTIVATIONS = {"silu": 1, None: 0}


def _conv_desc(x, weight, bias, activation, step):
    _cuda(x, "x")
    code = _code(x, "x")
    _need(x.dim() == (2 if step else 3), "x must have shape " + ("(batch, channels)" if step else
                                                                "(batch, length, channels)"))
    _like(x, "x", x.shape, x.dtype, x.device)
    _need(weight.dim() == 2 and 1 <= weight.shape[1] <= SC_CONV_MAX_WIDTH,
          "weight must have shape (channels, width), width 1 to %d" % SC_CONV_MAX_WIDTH)
    _need(activation in _ACTIVATIONS, "activation must be 'silu' or None")
    channels, width = x.shape[-1], weight.shape[1]
    import torch
    wp = _whole(weight, "weight", torch.Size((channels, width)), x.dtype, x.device)
    bp = _whole(bias, "bias", torch.Size((channels,)), x.dtype, x.device)
    return ConvDesc(dtype=code, width=width, silu=_ACTIVATIONS[activation], batch=x.shape[0],
                    length=1 if step else x.shape[1], channels=channels, x=x.data_ptr(), x_batch=x.stride(0),
                    x_token=0 if step else x.stride(1), weight=wp, bias=bp)


def _conv_extra(d, x, heads, state):
    import torch
    d.heads = _heads(heads, x.shape[:2], x.device)
    shape = torch.Size((d.batch, d.width - 1, d.channels))
    d.state = _whole(state, "state", shape, x.dtype, x.device)
    return shape


def causal_conv(x, weight, bias=None, activation="silu", heads=None, state=None, final_state=None, out=None,
                stream=None):
    """Causal convolution of x (batch, length, channels) with weight (channels,
    width), one filter per channel.  state: the width - 1 inputs before x, oldest
    first (batch, width - 1, channels); final_state: receives those after x."""
    import torch
    d = _conv_desc(x, weight, bias, activation, False)
    shape = _conv_extra(d, x, heads, state)
    fp = _whole(final_state, "final_state", shape, x.dtype, x.device)
    if out is None:
        with _on(stream):
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    else:
        _like(out, "out", x.shape, x.dtype, x.device)
    _check(_lib().sc_causal_conv(d, out.data_ptr(), out.stride(0), out.stride(1), fp, _stream(stream)),
           "sc_causal_conv")
    return out


def causal_conv_grad(dy, x, weight, bias=None, activation="silu", heads=None, state=None, stream=None):
    """Gradients of causal_conv: a dict with x (x's type), weight and bias (float32)
    and, where `state` is given, state (x's type)."""
    import torch
    d = _conv_desc(x, weight, bias, activation, False)
    shape = _conv_extra(d, x, heads, state)
    _like(dy, "dy", x.shape, x.dtype, x.device)
    with _on(stream):
        grads = {"x": torch.empty(x.shape, dtype=x.dtype, device=x.device),
                 "weight": torch.empty(weight.shape, dtype=torch.float32, device=x.device),
                 "bias": torch.empty(d.channels, dtype=torch.float32, device=x.device)}
        if state is not None:
            grads["state"] = torch.empty(shape, dtype=x.dtype, device=x.device)
    dx = grads["x"]
    _check(_lib().sc_causal_conv_grad(d, dy.data_ptr(), dy.stride(0), dy.stride(1), dx.data_ptr(), dx.stride(0),
                                      dx.stride(1), grads["weight"].data_ptr(), grads["bias"].data_ptr(),
                                      grads["state"].data_ptr() if state is not None else 0, _stream(stream)),
           "sc_causal_conv_grad")
    return grads


def _slots(slots, batch, device) -> int:
    import torch
    return _whole(slots, "slots", torch.Size((batch,)), torch.int32, device)


def causal_conv_step(x, state, weight, bias=None, activation="silu", slots=None, out=None, stream=None):
    """One token for each row of x (batch, channels); state (rows, width - 1,
    channels) is moved on in place.  slots (int32): the state row of each x row,
    no row twice; outside [0, rows): the x row sits out, its y is 0."""
    import torch
    d = _conv_desc(x, weight, bias, activation, True)
    _need(state.dim() == 3, "state must have shape (rows, width - 1, channels)")
    rows = state.shape[0]
    sp = _whole(state, "state", torch.Size((rows, d.width - 1, d.channels)), x.dtype, x.device)
    if out is None:
        with _on(stream):
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    else:
        _like(out, "out", x.shape, x.dtype, x.device)
    _check(_lib().sc_causal_conv_step(d, sp, rows, _slots(slots, d.batch, x.device), out.data_ptr(), out.stride(0),
                                      _stream(stream)), "sc_causal_conv_step")
    return out


# ---------------------------------------------------------- selective scan
def _ssm_desc(x, dt, A, B, C, D, z, dt_bias, softplus, step):
    import torch
    _cuda(x, "x")
    code = _code(x, "x")
    dtype, device = x.dtype, x.device
    _need(x.dim() == (2 if step else 3), "x must have shape " + ("(batch, channels)" if step else
                                                                "(batch, length, channels)"))
    _like(x, "x", x.shape, dtype, device)
    _like(dt, "dt", x.shape, dtype, device)
    channels = x.shape[-1]
    _need(A.dim() == 2 and 1 <= A.shape[1], "A must have shape (channels, states)")
    states = A.shape[1]
    ap = _whole(A, "A", torch.Size((channels, states)), torch.float32, device)
    _need(B.dim() == x.dim() + 1 and B.shape[-2] >= 1, "B must have shape (batch, length, groups, states)")
    groups = B.shape[-2]
    _need(channels % groups == 0, "channels must be a multiple of the groups of B and C")
    shape = x.shape[:-1] + (groups, states)
    _like(B, "B", shape, dtype, device)
    _like(C, "C", shape, dtype, device)
    if z is not None:
        _like(z, "z", x.shape, dtype, device)
    vec = torch.Size((channels,))
    bs, cs = B.stride(), C.stride()
    d = SsmDesc(dtype=code, softplus=int(softplus), batch=x.shape[0], length=1 if step else x.shape[1],
                channels=channels, states=states, groups=groups, x=x.data_ptr(), dt=dt.data_ptr(),
                x_batch=x.stride(0), dt_batch=dt.stride(0), A=ap, B=B.data_ptr(), C=C.data_ptr(), B_batch=bs[0],
                B_group=bs[-2], C_batch=cs[0], C_group=cs[-2],
                D=_whole(D, "D", vec, torch.float32, device), z=0 if z is None else z.data_ptr(),
                z_batch=0 if z is None else z.stride(0),
                dt_bias=_whole(dt_bias, "dt_bias", vec, torch.float32, device))
    if not step:
        d.x_token, d.dt_token, d.B_token, d.C_token = x.stride(1), dt.stride(1), bs[1], cs[1]
        d.z_token = 0 if z is None else z.stride(1)
    return d


def _saved_shape(batch, length, channels, states):
    padded = 8 if states <= 8 else 16 if states <= 16 else 32 if states <= 32 else 64
    return batch, -(-length // SC_SSM_SAVE), channels, padded


def selective_scan_saved(x, A, stream=None):
    """The buffer that a selective_scan of x with A fills for selective_scan_grad."""
    import torch
    with _on(stream):
        return torch.empty(_saved_shape(*x.shape, A.shape[1]), dtype=torch.float32, device=x.device)


def selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus: bool = True, heads=None, state=None,
                   final_state=None, saved=None, out=None, stream=None):
    """Selective state space scan of x (batch, length, channels): dt like x, A
    (channels, states) float32, B and C (batch, length, groups, states), D and
    dt_bias (channels) float32, z like x.  state / final_state: (batch, channels,
    states) float32.  saved: from selective_scan_saved, for the gradient."""
    import torch
    d = _ssm_desc(x, dt, A, B, C, D, z, dt_bias, softplus, False)
    dtype, device = x.dtype, x.device
    shape = torch.Size((d.batch, d.channels, d.states))
    d.heads = _heads(heads, x.shape[:2], device)
    d.state = _whole(state, "state", shape, torch.float32, device)
    fp = _whole(final_state, "final_state", shape, torch.float32, device)
    sp = _whole(saved, "saved", torch.Size(_saved_shape(d.batch, d.length, d.channels, d.states)), torch.float32, device)
    if out is None:
        with _on(stream):
            out = torch.empty(x.shape, dtype=dtype, device=device)
    else:
        _like(out, "out", x.shape, dtype, device)
    _check(_lib().sc_selective_scan(d, out.data_ptr(), out.stride(0), out.stride(1), fp, sp, _stream(stream)),
           "sc_selective_scan")
    return out


def selective_scan_grad(dy, x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus: bool = True, heads=None,
                        state=None, saved=None, dfinal_state=None, stream=None):
    """Gradients of selective_scan, given what it saved: a dict with x, dt, B, C
    (their types), A, and those of D, z, dt_bias and state that were given."""
    import torch
    d = _ssm_desc(x, dt, A, B, C, D, z, dt_bias, softplus, False)
    dtype, device = x.dtype, x.device
    shape = torch.Size((d.batch, d.channels, d.states))
    d.heads = _heads(heads, x.shape[:2], device)
    d.state = _whole(state, "state", shape, torch.float32, device)
    _like(dy, "dy", x.shape, dtype, device)
    _need(saved is not None, "saved: the buffer that selective_scan filled is needed")
    sp = _whole(saved, "saved", torch.Size(_saved_shape(d.batch, d.length, d.channels, d.states)), torch.float32, device)
    dfp = _whole(dfinal_state, "dfinal_state", shape, torch.float32, device)
    with _on(stream):
        g = {"x": torch.empty(x.shape, dtype=dtype, device=device), "dt": torch.empty(x.shape, dtype=dtype, device=device),
             "A": torch.empty(A.shape, dtype=torch.float32, device=device),
             "B": torch.empty(B.shape, dtype=dtype, device=device), "C": torch.empty(C.shape, dtype=dtype, device=device)}
        if D is not None:
            g["D"] = torch.empty(d.channels, dtype=torch.float32, device=device)
        if z is not None:
            g["z"] = torch.empty(x.shape, dtype=dtype, device=device)
        if dt_bias is not None:
            g["dt_bias"] = torch.empty(d.channels, dtype=torch.float32, device=device)
        if state is not None:
            g["state"] = torch.empty(shape, dtype=torch.float32, device=device)
    ptr = {k: v.data_ptr() for k, v in g.items()}
    out = SsmGrads(dy=dy.data_ptr(), dy_batch=dy.stride(0), dy_token=dy.stride(1), saved=sp, dfinal=dfp, dx=ptr["x"],
                   ddt=ptr["dt"], dz=ptr.get("z", 0), dB=ptr["B"], dC=ptr["C"], dA=ptr["A"], dD=ptr.get("D", 0),
                   ddt_bias=ptr.get("dt_bias", 0), dstate=ptr.get("state", 0))
    _check(_lib().sc_selective_scan_grad(d, out, _stream(stream)), "sc_selective_scan_grad")
    return g


def selective_scan_step(x, dt, A, B, C, state, D=None, z=None, dt_bias=None, softplus: bool = True, slots=None,
                        out=None, stream=None):
    """One token for each row of x (batch, channels), B and C (batch, groups,
    states); state (rows, channels, states) float32 is moved on in place.  slots
    as in causal_conv_step."""
    import torch
    d = _ssm_desc(x, dt, A, B, C, D, z, dt_bias, softplus, True)
    _need(state.dim() == 3, "state must have shape (rows, channels, states)")
    rows = state.shape[0]
    sp = _whole(state, "state", torch.Size((rows, d.channels, d.states)), torch.float32, x.device)
    if out is None:
        with _on(stream):
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    else:
        _like(out, "out", x.shape, x.dtype, x.device)
    _check(_lib().sc_selective_scan_step(d, sp, rows, _slots(slots, d.batch, x.device), out.data_ptr(), out.stride(0),
                                         _stream(stream)), "sc_selective_scan_step")
    return out
