"""The norm, the gated recurrence and the way to experts in float64, from their
definitions, each with a bound of the error of its float32 computation.

Every function returns pairs (value, bound) by name.  EPS = 2^-24, U the rounding unit
of an output's type (half a step), and a sum of terms t_i of depth D is off by at most
D EPS sum |t_i|.

Norm.  A row's sums are taken by up to 16 additions in a thread, 5 in a warp and 32
over warps, and beyond 8192 channels channels / 1024 in a thread: D = 64 + channels /
1024.  With M = mean |s|:
  dm  = (D + 2) EPS M                                      error of the mean
  dv  = (D + 4) EPS + 2 dm mean|c| / v + dm^2 / v          of the variance v, relative
  dr  = dv / 2 + 4 EPS                                     of r (sum with eps, root, quotient)
  dn  = |n| (dr + 2 EPS) + dm r                            of n = (s - m) r
  y: |w| dn + 2 EPS (|n w| + |b|).
Gradient, with dn as above (m and r are those that were saved), g = dy w:
  da  = (D + 2) EPS mean|g|,  db = (D + 4) EPS mean|g n| + mean(|g| dn)
  dx: r (da + |n| db + |b| dn + 6 EPS (|g| + |a| + |n b|)) + dr |dx| + EPS |dsum|
  dweight: sum |dy| dn + rows EPS sum |dy n|;  dbias: rows EPS sum |dy|.

Gated recurrence.  rest = 1 - f = e / (1 + e), e = exp(-g): the exponential's own error
of 4 EPS and, with 16-bit elements, |g| EPS of its argument; sum, reciprocal and product
4: rest is off by C = 8 + |g| <= 24 relative, and f = 1 - rest by C rest + 1 absolute, in
EPS.  Without the sigmoid both are exact.  With m the recurrence over absolute values
and F = C rest + 1 (0 without the sigmoid):
  eh[t] = f eh[t-1] + (F + 8 f) EPS m[t-1] + (C + 8) EPS |b[t]|,
where 8 covers the product and sum of a step and a step's share of the maps of whole
tiles (16 products and the like a tile); a tile's fold over warps and CTAs adds at most
2 EPS for each of up to 16 of them: 32 EPS m once.  Backwards the same:
  ed[t] = f ed[t+1] + (F + 8 f) EPS md[t+1], + 32 EPS md once.

Experts.  A token's sum of k terms: (k + 1) EPS sum |w y|; a product of dim elements:
(dim + 2) EPS sum |dout y|; products: EPS.
"""
import torch

EPS = 2.0 ** -24
UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}


def check(name, got, pair):
    """got within its bound, and its type's rounding, of the value."""
    want, bound = pair
    dtype = got.dtype
    got = got.detach().double().cpu()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    allowed = bound + UNIT[dtype] * (want.abs() + bound) + TINY[dtype]
    bad = ~((got - want).abs() <= allowed)
    assert not bad.any(), "%s: %d of %d outside, first %s: got %r want %r allowed %r" % (
        name, int(bad.sum()), bad.numel(), tuple(int(i) for i in bad.nonzero()[0]), got[bad][0].item(),
        want[bad][0].item(), allowed[bad][0].item())


# --------------------------------------------------------------------- norm
def norm(x, weight=None, bias=None, eps=1e-5, rms=False, residual=None, dy=None, dsum=None):
    """x (rows, channels); `dy`: also the gradients, with `dsum` added to x's."""
    ch = x.shape[-1]
    s = x.double() if residual is None else (x.float() + residual.float()).to(x.dtype).double()
    w = torch.ones(ch, dtype=torch.float64) if weight is None else weight.double()
    b = torch.zeros(ch, dtype=torch.float64) if bias is None else bias.double()

    def mean(t):
        return t.sum(-1, keepdim=True) / ch

    depth = 64 + ch / 1024
    m = torch.zeros_like(mean(s)) if rms else mean(s)
    dm = torch.zeros_like(m) if rms else (depth + 2) * EPS * mean(s.abs())
    c = s - m
    v = mean(c * c) + eps
    r = v ** -0.5
    dv = (depth + 4) * EPS + 2 * dm * mean(c.abs()) / v + dm * dm / v
    dr = dv / 2 + 4 * EPS
    n = c * r
    dn = n.abs() * (dr + 2 * EPS) + dm * r
    out = {"sum": (s, torch.zeros_like(s)), "mean": (m, dm), "r": (r, dr * r),
           "y": (n * w + b, w.abs() * dn + 2 * EPS * ((n * w).abs() + b.abs()))}
    if dy is None:
        return out
    d, rows = dy.double(), x.shape[0]
    g = d * w
    a = torch.zeros_like(m) if rms else mean(g)
    da = torch.zeros_like(m) if rms else (depth + 2) * EPS * mean(g.abs())
    q = mean(g * n)
    dq = (depth + 4) * EPS * mean((g * n).abs()) + mean(g.abs() * dn)
    dx = (g - a - n * q) * r
    bound = r * (da + n.abs() * dq + q.abs() * dn + 6 * EPS * (g.abs() + a.abs() + (n * q).abs())) + dr * dx.abs()
    if dsum is not None:
        bound = bound + EPS * (dsum.double().abs() + dx.abs())
        dx = dx + dsum.double()
    out["dx"] = (dx, bound)
    out["dweight"] = ((d * n).sum(0), (d.abs() * dn).sum(0) + rows * EPS * (d * n).abs().sum(0))
    out["dbias"] = (d.sum(0), rows * EPS * d.abs().sum(0))
    return out


# -------------------------------------------------------------------- gated
def gated(x, gate, activation="sigmoid", heads=None, state=None, dy=None, dfinal=None):
    """x and gate (batch, length, channels)."""
    batch, length, ch = x.shape
    x, g = x.double(), gate.double()
    if activation is None:
        f, rest, C = g, torch.ones_like(g), 0.0
    else:
        f, rest, C = 1 / (1 + torch.exp(-g)), 1 / (1 + torch.exp(g)), 24.0
        assert g.abs().max() <= 16 if g.numel() else True
    keep = torch.ones(batch, length, 1, dtype=torch.bool) if heads is None else ~heads.bool()[:, :, None]
    zero = torch.zeros(batch, ch, dtype=torch.float64)
    h = zero if state is None else state.double()
    m, e = h.abs(), zero
    y, ey, before, mb, eb = [], [], [], [], []
    for t in range(length):
        h, m, e = (torch.where(keep[:, t], v, 0.0) for v in (h, m, e))
        before.append(h)
        mb.append(m)
        eb.append(e)
        b = rest[:, t] * x[:, t]
        ft = torch.where(keep[:, t], f[:, t], 0.0)
        off = torch.where(keep[:, t], (C * rest[:, t] + 1 if C else 0.0) + 8 * ft.abs(), 0.0)  # of f, and a step's roundings
        e = ft.abs() * e + EPS * (off * m + (C + 8) * b.abs())
        h = ft * h + b
        m = ft.abs() * m + b.abs()
        y.append(h)
        ey.append(e + 32 * EPS * m)
    stack = lambda v: torch.stack(v, 1) if v else torch.zeros(batch, 0, ch, dtype=torch.float64)  # noqa: E731
    out = {"y": (stack(y), stack(ey)), "final": (h, e + 32 * EPS * m)}
    if dy is None:
        return out
    d = dy.double()
    q = zero if dfinal is None else dfinal.double()
    mq, eq = q.abs(), zero
    dx, edx, dg, edg = [], [], [], []
    for t in reversed(range(length)):
        dh, mh = d[:, t] + q, d[:, t].abs() + mq
        eh = eq + EPS * mh + 32 * EPS * mh
        w = rest[:, t]
        dx.append(dh * w)
        edx.append((eh + (C + 2) * EPS * dh.abs()) * w)
        if activation is None:
            u, scale, mu = before[t], torch.ones_like(w), mb[t]
            eu = eb[t]
        else:
            u, scale, mu = before[t] - x[:, t], f[:, t] * w, mb[t] + x[:, t].abs()
            eu = eb[t] + EPS * mu
        dg.append(dh * u * scale)
        # f and rest in dgate: rest's error relative, f's absolute
        edg.append((eh * u.abs() + dh.abs() * (eu + 32 * EPS * mu) + (C + 8) * EPS * (dh * u).abs()) * scale
                   + ((C * w + 1) * w * EPS * (dh * u).abs() if C else 0.0))
        ft = torch.where(keep[:, t], f[:, t], 0.0).abs()
        live = keep[:, t]
        off = torch.where(live, (C * w + 1 if C else 0.0) + 8 * ft, 0.0)
        eq = ft * (eq + EPS * mh) + off * EPS * mh
        q, mq = torch.where(live, f[:, t], 0.0) * dh, ft * mh
    rev = lambda v: stack(v[::-1])  # noqa: E731
    return out | {"dx": (rev(dx), rev(edx)), "dgate": (rev(dg), rev(edg)), "dstate": (q, eq + 32 * EPS * mq)}


# ------------------------------------------------------------------ experts
def expert_sort(ids, experts):
    """offsets, order and place as lists."""
    bins = [[] for _ in range(experts + 1)]
    for entry, expert in enumerate(ids.flatten().tolist()):
        bins[expert if 0 <= expert < experts else experts].append(entry)
    order = [e for b in bins for e in b]
    offsets = [0]
    for b in bins[:experts]:
        offsets.append(offsets[-1] + len(b))
    place = [0] * len(order)
    for row, entry in enumerate(order):
        place[entry] = row
    return offsets, order, place


def expert_rows(x, order, offsets, choices):
    """The gathered rows, exact."""
    rows = torch.zeros(len(order), x.shape[1], dtype=x.dtype)
    kept = offsets[-1]
    if kept:
        rows[:kept] = x[torch.tensor(order[:kept]) // choices]
    return rows


def expert_combine(y, place, kept, tokens, choices, weights=None, dout=None):
    """The token's sums, and with `dout` the gradients by y and by the weights."""
    dim = y.shape[1]
    total, size = torch.zeros(tokens, dim, dtype=torch.float64), torch.zeros(tokens, dim, dtype=torch.float64)
    dy, dw, dws = torch.zeros(y.shape, dtype=torch.float64), *(torch.zeros(tokens, choices, dtype=torch.float64),) * 2
    dws = torch.zeros_like(dw)
    place = torch.tensor(place, dtype=torch.int64).view(tokens, choices)
    for j in range(choices):
        live = place[:, j] < kept
        at = place[live, j]
        w = torch.ones(int(live.sum()), 1, dtype=torch.float64) if weights is None else weights.double()[live, j, None]
        rows = y[at].double()
        total[live] += w * rows
        size[live] += (w * rows).abs()
        if dout is not None:
            d = dout.double()[live]
            dy[at] = w * d
            dw[live, j] = (d * rows).sum(1)
            dws[live, j] = (d * rows).abs().sum(1)
    out = {"out": (total, (choices + 1) * EPS * size)}
    if dout is not None:
        out |= {"dy": (dy, EPS * dy.abs()), "dweights": (dw, (dim + 2) * EPS * dws)}
    return out
