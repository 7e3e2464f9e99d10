"""The sequence operators in float64, token by token, from their definitions, and
the error bounds of their float32 computation.

Bounds.  EPS = 2^-24.  Every output is a sum of products of computed factors.
Let `c` bound the relative error of one factor in units of EPS:

* d = softplus(dt + bias): the sum's rounding is |v| EPS in v and as much,
  relatively, in d (|v d'(v)| <= |v| d); the function adds 4; |v| <= 8 in the
  tests: 12;
* exp(d A): the exponent's relative error (12 + 3) times |d A|, and the
  instruction's 4: 4 + 15 |d A|, |d A| <= 8 where the factor still counts
  (beyond, it is below 4e-4 of its neighbours' terms and its error below 2e-2 of
  that): 124;
* products, activations (8 with their argument's error <= 8 more): 16.

C_FACTOR = 128 covers each.  A term of an output at length L has at most
2 L + 8 such factors (the decays forth and back, and the rest), and a float32
sum of m terms in any order adds m roundings, so

    |got - want| <= U |want| + (2 L + 8) C_FACTOR EPS M + m EPS M

with U the rounding unit of the output's type (plus its smallest subnormal) and
M the same sum over absolute values.  The bounds are worst cases: an error of
the formula (a missing term, a wrong index, a state of the wrong token) is of
the size of M itself.
"""
import torch

EPS = 2.0 ** -24
C_FACTOR = 128
UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}


def check(name, got, want, magnitude, dtype, length, terms):
    """got within the bound of the module's docstring."""
    got, want, magnitude = got.double().cpu(), want.double().cpu(), magnitude.double().cpu()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    bound = UNIT[dtype] * want.abs() + TINY[dtype] + ((2 * length + 8) * C_FACTOR + terms) * EPS * magnitude
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), "%s: %d of %d outside, first %s: got %r want %r bound %r" % (
        name, int(bad.sum()), bad.numel(), tuple(int(i) for i in bad.nonzero()[0]), got[bad][0].item(),
        want[bad][0].item(), bound[bad][0].item())


def silu(v):
    return v / (1 + torch.exp(-v))


def dsilu(v):
    s = 1 / (1 + torch.exp(-v))
    return s + v * s * (1 - s)


# ---------------------------------------------------------------- embedding
def embed(ids, weight, scale):
    out = torch.zeros(ids.numel(), weight.shape[1], dtype=torch.float64)
    for t, i in enumerate(ids.reshape(-1).tolist()):
        if 0 <= i < weight.shape[0]:
            out[t] = weight[i].double() * scale
    return out.reshape(*ids.shape, weight.shape[1])


def embed_grad(ids, dout, vocab, scale):
    """The sums, the sums of absolute values, and how many terms each row has."""
    rows = dout.double().reshape(-1, dout.shape[-1])
    flat = ids.reshape(-1).long()
    keep = (flat >= 0) & (flat < vocab)
    total = torch.zeros(vocab, dout.shape[-1], dtype=torch.float64)
    size = torch.zeros_like(total)
    total.index_add_(0, flat[keep], rows[keep] * scale)
    size.index_add_(0, flat[keep], (rows[keep] * scale).abs())
    return total, size, torch.bincount(flat[keep], minlength=vocab)


# -------------------------------------------------------------- convolution
def conv(x, weight, bias, heads=None, state=None, act=True, dy=None):
    """y, final state, and the gradients for dy; each with its sum of absolute
    values where it is a sum."""
    x, w = x.double(), weight.double()
    batch, length, ch = x.shape
    width = w.shape[1]
    before = torch.zeros(batch, width - 1, ch, dtype=torch.float64) if state is None else state.double()
    line = torch.cat([before, x], 1)
    r = {"pre": torch.zeros_like(x), "size": torch.zeros_like(x)}
    begin = torch.full((batch,), -width)
    sees = torch.zeros(batch, length, width)
    for t in range(length):
        if heads is not None:
            begin = torch.where(heads[:, t] != 0, torch.full_like(begin, t), begin)
        r["pre"][:, t] = 0 if bias is None else bias.double()
        r["size"][:, t] = r["pre"][:, t].abs()
        for k in range(width):
            on = (t - (width - 1 - k) >= begin)
            sees[:, t, k] = on
            term = torch.where(on[:, None], w[:, k] * line[:, t + k], 0.0)
            r["pre"][:, t] += term
            r["size"][:, t] += term.abs()
    r["y"] = silu(r["pre"]) if act else r["pre"].clone()
    final = line[:, length:].clone()
    for j in range(width - 1):
        final[:, j][length - (width - 1) + j < begin] = 0
    r["final"] = final
    if dy is None:
        return r
    slope = dsilu(r["pre"]) if act else torch.ones_like(x)
    # the slope's error: that of pre times the second derivative (at most 1/2)
    dpre = dy.double() * slope
    size = dy.double().abs() * (slope.abs() + r["size"])
    dline, dsize = torch.zeros_like(line), torch.zeros_like(line)
    dw, wsize = torch.zeros_like(w), torch.zeros_like(w)
    for t in range(length):
        for k in range(width):
            on = sees[:, t, k][:, None].bool()
            dline[:, t + k] += torch.where(on, w[:, k] * dpre[:, t], 0.0)
            dsize[:, t + k] += torch.where(on, w[:, k].abs() * size[:, t], 0.0)
            dw[:, k] += torch.where(on, dpre[:, t] * line[:, t + k], 0.0).sum(0)
            wsize[:, k] += torch.where(on, size[:, t] * line[:, t + k].abs(), 0.0).sum(0)
    r |= {"dx": dline[:, width - 1:], "dx_size": dsize[:, width - 1:], "dstate": dline[:, :width - 1],
          "dstate_size": dsize[:, :width - 1], "dweight": dw, "dweight_size": wsize, "dbias": dpre.sum((0, 1)),
          "dbias_size": size.sum((0, 1))}
    return r


# ----------------------------------------------------------- selective scan
def scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus=True, heads=None, state=None, dy=None, dfinal=None,
         sizes=False):
    """y, final state and, for dy, the gradients.  sizes: every product by its
    absolute value (the decays are positive), which gives each output's M."""
    f = (lambda v: v.double().abs()) if sizes else (lambda v: v.double())
    batch, length, ch = x.shape
    n, groups = A.shape[1], B.shape[2]
    per = ch // groups
    v = dt.double() + (0 if dt_bias is None else dt_bias.double())
    d = torch.nn.functional.softplus(v, threshold=700) if softplus else v
    slope = torch.sigmoid(v) if softplus else torch.ones_like(v)
    x, rate = f(x), A.double()
    B = f(B).repeat_interleave(per, 2)
    C = f(C).repeat_interleave(per, 2)
    skip = torch.zeros(ch, dtype=torch.float64) if D is None else f(D)
    first = torch.zeros(batch, ch, n, dtype=torch.float64) if state is None else f(state)
    dabs = d.abs() if sizes else d
    h, hs, qs = first, [], []
    y0 = torch.zeros_like(x)
    for t in range(length):
        q = torch.exp(d[:, t, :, None] * rate)
        if heads is not None:
            q = torch.where((heads[:, t] != 0)[:, None, None], 0.0, q)
            h = torch.where((heads[:, t] != 0)[:, None, None], 0.0, h)
        h = q * h + (dabs[:, t] * x[:, t])[..., None] * B[:, t]
        hs.append(h)
        qs.append(q)
        y0[:, t] = (C[:, t] * h).sum(-1) + skip * x[:, t]
    zd = None if z is None else z.double()
    gate = torch.ones_like(x) if z is None else (silu(zd).abs() if sizes else silu(zd))
    r = {"y": y0 * gate, "final": h}
    if dy is None:
        return r
    g = f(dy) * gate
    if z is not None:
        r["dz"] = f(dy) * y0 * (dsilu(zd).abs() if sizes else dsilu(zd))
    per_group = lambda u: u.unflatten(1, (groups, per)).sum(2)  # noqa: E731
    dh = torch.zeros(batch, ch, n, dtype=torch.float64) if dfinal is None else f(dfinal)
    dx, dd, dA = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(rate)
    dB, dC = (torch.zeros(batch, length, groups, n, dtype=torch.float64) for _ in range(2))
    for t in reversed(range(length)):
        dh = dh + C[:, t] * g[:, t, :, None]
        dC[:, t] = per_group(g[:, t, :, None] * hs[t])
        dB[:, t] = per_group(dh * (dabs[:, t] * x[:, t])[..., None])
        back = dh * qs[t]
        before = hs[t - 1] if t else first
        if heads is not None:
            before = torch.where((heads[:, t] != 0)[:, None, None], 0.0, before)
        by_exponent = back * before
        dhb = (dh * B[:, t]).sum(-1)
        dA += (by_exponent * dabs[:, t, :, None]).sum(0)
        dd[:, t] = (by_exponent * (rate.abs() if sizes else rate)).sum(-1) + dhb * x[:, t]
        dx[:, t] = dhb * dabs[:, t] + skip * g[:, t]
        dh = back
    dv = dd * slope
    r |= {"dx": dx, "ddt": dv, "dA": dA, "dB": dB, "dC": dC, "dD": (g * x).sum((0, 1)), "ddt_bias": dv.sum((0, 1)),
          "dstate": dh}
    return r
