"""Numbers of states that the kernels pad (anything but 8, 16, 32 and 64): an infinity
among the elements gives what the definition gives, not infinity times a padded zero."""
import pytest
import torch

import seq_reference as ref
import stream_compaction_gb300 as sc
from gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def _case(length, states, channels=20, dtype=torch.float32, batch=1, groups=1):
    """Everything positive but A, so that an infinity stays one in every sum.  |d A| is at
    most 0.2 (no decay underflows, but where d itself is infinite)."""
    gen = torch.Generator().manual_seed(length + states)

    def positive(*shape, dtype=dtype):
        return (0.5 + torch.rand(*shape, generator=gen)).to(dtype)

    c = {"x": positive(batch, length, channels), "dt": (positive(batch, length, channels) / 10).to(dtype),
         "A": -positive(channels, states, dtype=torch.float32), "B": positive(batch, length, groups, states),
         "C": positive(batch, length, groups, states), "D": positive(channels, dtype=torch.float32),
         "state": positive(batch, channels, states, dtype=torch.float32)}
    return c, positive(batch, length, channels)


def _same(name, got, want):
    """The same infinities and NaN, and numbers as close as float32 sums of positive terms are."""
    got, want = got.double().cpu(), want.double()
    assert torch.equal(got.isnan(), want.isnan()), (name, "NaN")
    assert torch.equal(got.isinf(), want.isinf()) and torch.equal(got[got.isinf()], want[want.isinf()]), name
    rest = torch.isfinite(want)
    # no cancellation: 128 units a factor (seq_reference), up to 400 of them; 16 bits: their rounding
    assert torch.allclose(got[rest], want[rest], rtol=400 * 128 * 2.0 ** -24 + 2.0 ** -8, atol=0), name


def _run(c, dy):
    d = {k: v.cuda() for k, v in c.items()}
    final = torch.empty_like(d["state"])
    saved = sc.selective_scan_saved(d["x"], d["A"])
    y = sc.selective_scan(**d, softplus=False, final_state=final, saved=saved)
    alone = torch.empty_like(d["state"])
    assert torch.equal(sc.selective_scan(**d, softplus=False, final_state=alone).isnan(), y.isnan())
    assert torch.equal(final.isnan(), alone.isnan())
    return y, final, sc.selective_scan_grad(dy.cuda(), **d, softplus=False, saved=saved)


def _check(c, dy, names):
    y, final, g = _run(c, dy)
    r = ref.scan(**c, softplus=False, dy=dy)
    _same("y", y, r["y"])
    _same("final", final, r["final"])
    for name in names:
        _same(name, g[name], r[{"x": "dx", "state": "dstate", "D": "dD", "B": "dB", "C": "dC"}[name]])


STATES = [1, 3, 6, 8, 12, 16, 24, 33, 60]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("length", [5, 37, 400])
@pytest.mark.parametrize("states", STATES)
def test_an_infinite_input(states, length, dtype):
    """Alone from its token on; a later segment start clears it.  Length 400: in chunks."""
    c, dy = _case(length, states, dtype=dtype)
    c["x"][0, 2, 3] = INF
    _check(c, dy, ["x", "state", "D", "B", "C"])
    c["heads"] = torch.zeros(1, length, dtype=torch.bool)
    c["heads"][0, 4] = True
    _check(c, dy, ["x", "state", "D", "B", "C"])


@pytest.mark.parametrize("length", [5, 37, 400])
@pytest.mark.parametrize("states", STATES)
def test_an_infinite_step(states, length):
    c, dy = _case(length, states)
    c["dt"][0, 2, 3] = INF
    _check(c, dy, ["state", "D", "C"])


@pytest.mark.parametrize("length", [5, 37, 400])
@pytest.mark.parametrize("states", STATES)
def test_an_infinite_gradient(states, length):
    c, dy = _case(length, states)
    dy[0, length - 2, 3] = INF
    _check(c, dy, ["x", "state", "D", "B", "C"])
    if length > 100:  # before a segment start, in chunks before, it is not seen
        c["heads"] = torch.zeros(1, length, dtype=torch.bool)
        c["heads"][0, length - 20] = True
        _, _, g = _run(c, dy)
        dy[0, length - 20:] = 0  # (the reference multiplies a decay of 0 by what comes from behind the start)
        r = ref.scan(**c, softplus=False, dy=dy)
        for name, of in (("x", "dx"), ("B", "dB"), ("C", "dC")):
            _same(name, g[name][:, :length - 20], r[of][:, :length - 20])
        _same("state", g["state"], r["dstate"])


@pytest.mark.parametrize("states", STATES)
def test_one_token(states):
    c, _ = _case(1, states, batch=5)
    c["x"][1, 0, 3] = c["dt"][2, 0, 4] = INF
    r = ref.scan(**c, softplus=False)
    d = {k: v.cuda() for k, v in c.items()}
    one = {k: d[k][:, 0] for k in ("x", "dt", "B", "C")}
    y = sc.selective_scan_step(**one, A=d["A"], D=d["D"], state=d["state"], softplus=False)
    _same("y", y, r["y"][:, 0])
    _same("state", d["state"], r["final"])
