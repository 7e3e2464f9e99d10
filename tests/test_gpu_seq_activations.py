"""Softplus and sigmoid inside the sequence operators' float32 forms, each isolated by
factors of one, against float64: relative errors in units of 2^-24.

Bounds, from the instructions' documented errors (2^t: 4 units, reciprocal: 2) and one
unit a rounding: exp(-|v|) 5; softplus = 2 artanh(e / (2 + e)): 5 + 1 + 2 + 1 for the
quotient, 2 more for the polynomial: 11, with 0.4 of the polynomial itself 12; sigmoid:
1 + e 1 (and at most half of e's), reciprocal 2, the product with e 1: 9; times v: 10.
"""
import pytest
import torch

import stream_compaction_gb300 as sc
from gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** -24
ROWS, CH = 64, 2048
RANGES = [(-87, -64), (-64, -32), (-32, -16), (-16, -8), (-8, -4), (-4, -2), (-2, 0), (0, 2), (2, 8), (8, 87)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def _values(lo, hi):
    gen = torch.Generator(device="cuda").manual_seed(hi - lo)
    return lo + (hi - lo) * torch.rand(ROWS, CH, generator=gen, device="cuda")


def _softplus(v):
    return v.clamp(min=0).double() + torch.log1p(torch.exp(-v.double().abs()))


def _sigmoid(v):
    e = torch.exp(-v.double().abs())
    return torch.where(v < 0, e, 1.0) / (1 + e)


def _within(got, want, units):
    off = ((got.double() - want).abs() / want.abs()).max().item() / UNIT
    assert off <= units, off


def _ones(*shape):
    return torch.ones(*shape, device="cuda")


@pytest.mark.parametrize("lo,hi", RANGES)
def test_softplus(lo, hi):
    v = _values(lo, hi)
    A, bc = -_ones(CH, 1), _ones(ROWS, 1, 1, 1)
    # one token, one state: y = C d x B = d
    y = sc.selective_scan(_ones(ROWS, 1, CH), v[:, None].contiguous(), A, bc, bc)
    _within(y[:, 0], _softplus(v), 12)
    y = sc.selective_scan_step(_ones(ROWS, CH), v, A, bc[:, 0], bc[:, 0], torch.zeros(ROWS, CH, 1, device="cuda"))
    _within(y, _softplus(v), 12)


@pytest.mark.parametrize("lo,hi", RANGES)
def test_sigmoid(lo, hi):
    v = _values(lo, hi)
    want = v.double() * _sigmoid(v)
    one = _ones(CH, 1)
    _within(sc.causal_conv(v[None].contiguous(), one)[0], want, 10)
    _within(sc.causal_conv_step(v, torch.empty(ROWS, 0, CH, device="cuda"), one), want, 10)
    x, bc = _ones(ROWS, 1, CH), _ones(ROWS, 1, 1, 1)
    saved = sc.selective_scan_saved(x, -one)
    # d = 1: y = z sigmoid(z)
    z = v[:, None].contiguous()
    _within(sc.selective_scan(x, x, -one, bc, bc, z=z, softplus=False)[:, 0], want, 10)
    y = sc.selective_scan_step(x[:, 0], x[:, 0], -one, bc[:, 0], bc[:, 0], torch.zeros(ROWS, CH, 1, device="cuda"), z=v,
                               softplus=False)
    _within(y, want, 10)
    # the gradient by dt: dd = 1, times the softplus's slope
    sc.selective_scan(x, z, -one, bc, bc, saved=saved)
    _within(sc.selective_scan_grad(x, x, z, -one, bc, bc, saved=saved)["dt"][:, 0], _sigmoid(v), 9)

def test_ends_and_what_is_no_number():
    inf, nan = float("inf"), float("nan")
    v = torch.tensor([[inf, 1e38, 3.4e38, 200.0, -200.0, -3.4e38, -inf, nan]], device="cuda")
    one, bc = _ones(8, 1), _ones(1, 1, 1)
    y = sc.selective_scan_step(_ones(1, 8), v, -one, bc, bc, torch.zeros(1, 8, 1, device="cuda"))[0]
    y2 = sc.selective_scan(_ones(1, 1, 8), v[:, None], -one, bc[None], bc[None])[0, 0]
    for got in (y, y2):
        assert got[0] == inf and torch.equal(got[1:4], v[0, 1:4]) and (got[4:7] == 0).all() and got[7].isnan()
    y = sc.causal_conv(v[None], one)[0, 0]
    assert y[0] == inf and torch.equal(y[1:4], v[0, 1:4]) and (y[4:6] == 0).all() and y[7].isnan()
