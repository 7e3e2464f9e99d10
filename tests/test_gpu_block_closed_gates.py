"""The gated recurrence where gates are nearly closed: f is small there, and what it
multiplies (a carried state, a gradient on its way back, the gate's own gradient) has f's
relative error.

Bounds, in EPS = 2^-24.  With e = exp(-|g|), the smaller of f and 1 - f, e / (1 + e), is off
by C = 8 + |g| relative: the exponential 4 and, with 16-bit elements, |g| of its argument;
sum, reciprocal and product 4.  The larger is 1 minus that: off by C + 1 relative at most.
With m the recurrence over absolute values, 8 for a step's product, sum and share of the
maps of whole tiles, and 32 m once for the fold of tiles over warps and CTAs:
  eh[t] = f (eh[t-1] + (C + 9) EPS m[t-1]) + (C + 9) EPS |b[t]|,   of h: eh + 32 EPS m
  eq[t] = f (eq[t+1] + (C + 9) EPS mq[t+1]),                       of dh: eq + 34 EPS mq
  dx = dh (1 - f):            (error of dh + (C + 3) EPS |dh|) (1 - f)
  dgate = dh (h - x) f (1 - f):
      (error of dh |u| + |dh| error of u + (2 C + 6) EPS |dh u|) f (1 - f),  u = h - x
Values below 2^-126 lose digits: FLOOR times what they are multiplied with.  Such a product
is a multiple of 2^-149, half a step of it off: u f (1 - f) by 2^-150, which dh multiplies
(float32: 7 steps of 2^-149 came out as 6, u f (1 - f) being a few steps itself).
"""
import pytest
import torch

import stream_compaction_gb300 as sc
from block_reference import EPS, UNIT, check
from gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu

FLOOR = 2.0 ** -124
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def _reference(x, gate, state, dy, dfinal):
    x, g, d = x.double(), gate.double(), dy.double()
    f, rest, C = 1 / (1 + torch.exp(-g)), 1 / (1 + torch.exp(g)), 8 + g.abs()
    b = rest * x
    h, m, e = state.double(), state.double().abs(), torch.zeros_like(state.double())
    ys, eys, us, eus, mus = [], [], [], [], []
    for t in range(x.shape[1]):
        off = (C[:, t] + 9) * EPS
        us.append(h - x[:, t])
        mus.append(m + x[:, t].abs())
        eus.append(e + 32 * EPS * m + 2 * EPS * mus[-1] + FLOOR)
        e = f[:, t] * (e + off * m) + off * b[:, t].abs()
        h, m = f[:, t] * h + b[:, t], f[:, t] * m + b[:, t].abs()
        ys.append(h)
        eys.append(e + 32 * EPS * m + FLOOR)
    q = dfinal.double()
    mq, eq = q.abs(), torch.zeros_like(q)
    dxs, edxs, dgs, edgs = [], [], [], []
    for t in reversed(range(x.shape[1])):
        dh, mh = d[:, t] + q, d[:, t].abs() + mq
        eh, w, c = eq + 34 * EPS * mh + FLOOR, rest[:, t], C[:, t]
        dxs.append(dh * w)
        edxs.append((eh + (c + 3) * EPS * dh.abs()) * w)
        dgs.append(dh * us[t] * f[:, t] * w)
        edgs.append((eh * us[t].abs() + dh.abs() * eus[t] + eh * eus[t] + (2 * c + 6) * EPS * (dh * us[t]).abs()) * f[:, t] * w
                    + FLOOR * (dh * us[t]).abs() + 2.0 ** -150 * dh.abs())
        eq = f[:, t] * (eq + EPS * mh + (c + 9) * EPS * mh)
        q, mq = f[:, t] * dh, f[:, t] * mh
    stack = lambda v: torch.stack(v, 1)  # noqa: E731
    return {"y": (stack(ys), stack(eys)), "final": (h, e + 32 * EPS * m + FLOOR), "dx": (stack(dxs[::-1]), stack(edxs[::-1])),
            "dgate": (stack(dgs[::-1]), stack(edgs[::-1])), "dstate": (q, eq + 34 * EPS * mq + FLOOR)}


def _case(batch, length, channels, dtype, often):
    """Open gates, and with probability `often` one from -30 to -8; the state is all that there is at first."""
    gen = torch.Generator().manual_seed(length + channels)
    u = torch.rand(3, batch, length, channels, generator=gen)
    g = torch.where(u[0] < often, -30 + 22 * u[1], 2 + 10 * u[2]).to(dtype)
    x = torch.zeros(batch, length, channels)
    x[:, length // 2:] = torch.randn(batch, length - length // 2, channels, generator=gen) * 1e-3
    dy = torch.randn(batch, length, channels, generator=gen).to(dtype)
    state, dfinal = (torch.randn(batch, channels, generator=gen) * 1e4 for _ in range(2))
    return x.to(dtype), g, state, dy, dfinal


def _check(name, got, pair):
    """As check; a value of half a step beyond the type's largest or more rounds to infinity
    (float16: 65520; what the states and gradients of 10^4 here multiply to passes it), so an
    infinity of the value's sign is right where the value and its bound reach that."""
    want, bound = pair
    info = torch.finfo(got.dtype)
    edge = info.max * (1 + UNIT[got.dtype] / 2)
    flat = got.detach().double().cpu()
    beyond = flat.isinf() & (flat.sign() == want.sign()) & (want.abs() + bound >= edge)
    keep = ~beyond
    check(name, got.detach().cpu()[keep], (want[keep], bound[keep]))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("often", [0.05, 1.0])
@pytest.mark.parametrize("batch,length,channels", [(2, 1, 64), (2, 40, 64), (1, 33, 37), (3, 50, 66), (1, 700, 128), (1, 645, 35)])
def test_carried_states_and_gradients(batch, length, channels, often, dtype):
    x, g, state, dy, dfinal = case = _case(batch, length, channels, dtype, often)
    r = _reference(*case)
    x, g, state, dy, dfinal = (t.cuda() for t in case)
    final, saved = torch.empty_like(state), sc.gated_scan_saved(x)
    y = sc.gated_scan(x, g, state=state, final_state=final, saved=saved)
    grads = sc.gated_scan_grad(dy, x, g, state=state, saved=saved, dfinal_state=dfinal)
    for name, t in (("y", y), ("final", final), ("dx", grads["x"]), ("dgate", grads["gate"]), ("dstate", grads["state"])):
        _check(name, t, r[name])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("channels", [64, 37])
def test_one_token(channels, dtype):
    x, g, state, dy, dfinal = case = _case(5, 1, channels, dtype, 1.0)
    r = _reference(*case)
    pool = state.cuda()
    y = sc.gated_scan_step(x[:, 0].cuda(), g[:, 0].cuda(), pool)
    check("y", y, tuple(v[:, 0] for v in r["y"]))
    check("pool", pool, r["final"])


@pytest.mark.parametrize("dtype", DTYPES)
def test_gates_without_end(dtype):
    """Gates of plus and minus infinity: exactly the old state, exactly x, whatever their sizes."""
    x = torch.full((1, 20, 64), 3.0, dtype=dtype, device="cuda")
    g = torch.full((1, 20, 64), float("inf"), dtype=dtype, device="cuda")
    state = torch.full((1, 64), 1e38, device="cuda")
    final, saved = torch.empty_like(state), sc.gated_scan_saved(x)
    sc.gated_scan(x, g, state=state, final_state=final, saved=saved)
    assert (final == state).all()
    grads = sc.gated_scan_grad(torch.ones_like(x), x, g, state=state, saved=saved)
    assert (grads["x"] == 0).all() and (grads["gate"] == 0).all() and (grads["state"] == 20).all()
    g = -g
    assert (sc.gated_scan(x, g, state=state, final_state=final, saved=saved) == 3).all() and (final == 3).all()
    grads = sc.gated_scan_grad(torch.ones_like(x), x, g, state=state, saved=saved)
    assert (grads["x"] == 1).all() and (grads["gate"] == 0).all() and (grads["state"] == 0).all()
