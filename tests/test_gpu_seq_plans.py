"""The plans that large problems run: chunks of many tiles and runs of several in the
scan's gradient, long runs in the convolution.  Every case first asserts the plan that it
is there for, from the workspace's size.

Besides the worst-case bounds of seq_reference, errors by norm: |got - want| against
|want| over the whole tensor, where a token lost at a join, a state rounded to 16 bits or
a partial sum left out cannot hide.  SMALL: states remember up to 400 tokens here (d of
0.05 times rates from 0.1); the decays' independent errors, 1.5 x 2^-24 each, add up to
sqrt(400) of it, 1.8e-6, and their mean error, at most 1.6e-8, to 400 / 2 of it, 3.2e-6.
Outputs in 16 bits: their own rounding besides, at most 0.6 units of roundoff by norm
(a uniform error over a uniform or logarithmic mantissa: 0.41 to 0.58)."""
import pytest
import torch

import seq_reference as ref
import stream_compaction_gb300 as sc
from gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu

SMALL = 5e-6
ROUNDING = {torch.float32: 0.0, torch.bfloat16: 0.6 * ref.UNIT[torch.bfloat16], torch.float16: 0.6 * ref.UNIT[torch.float16]}
WORKSPACE_HEAD = 4096  # in front of the scratch of these operators


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def _near(name, got, want, small=SMALL):
    off = ((got.double() - want.double()).norm() / want.double().norm()).item()
    assert off <= small + ROUNDING[got.dtype], (name, off)


# ------------------------------------------------------------ selective scan
def _padded(n):
    return (n + 255) // 256 * 256


def _scan_plan(batch, length, channels, states, groups):
    """(chunks, runs) of the gradient, from what its workspace holds."""
    lanes = 2 if states <= 8 else 4 if states <= 16 else 8 if states <= 32 else 16
    rows, np = {2: 128, 4: 128, 8: 64, 16: 16}[lanes], 4 * lanes
    blocks, tiles = -(-(channels // groups) // rows) * groups, -(-length // sc.SC_SSM_SAVE)
    total = sc.load().sc_selective_scan_grad_workspace_bytes(batch, length, channels, states, groups) - WORKSPACE_HEAD
    found = []
    for chunks in range(1, tiles + 1):
        for runs in range(chunks, tiles + 1) if chunks > 1 else [1]:
            size = _padded(blocks * batch * length * 2 * np * 4) + _padded(batch * chunks * channels * np * 4) + \
                _padded(2 * batch * chunks * channels * 4)
            if chunks > 1:
                size += _padded(batch * runs * channels * np * 4) + _padded(batch * runs * channels * 4) + _padded(batch * runs)
            if states != np:
                size += _padded(batch * chunks * blocks)
            if size == total:
                found.append((chunks, runs))
    assert len(found) == 1, found
    return found[0]


def _scan_case(batch, length, channels, states, groups, dtype, packed):
    gen = torch.Generator(device="cuda").manual_seed(length + channels + states)

    def normal(*shape, dtype=dtype, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    c = {"x": normal(batch, length, channels), "dt": normal(batch, length, channels, scale=0.3),
         "A": -(0.1 + 7.9 * torch.rand(channels, states, generator=gen, device="cuda")),
         "B": normal(batch, length, groups, states), "C": normal(batch, length, groups, states),
         "D": normal(channels, dtype=torch.float32), "z": normal(batch, length, channels),
         "dt_bias": normal(channels, dtype=torch.float32, scale=0.5) - 3,
         "state": normal(batch, channels, states, dtype=torch.float32)}
    if packed:
        c["heads"] = torch.rand(batch, length, generator=gen, device="cuda") < 1 / 150
    return c, normal(batch, length, channels), normal(batch, channels, states, dtype=torch.float32)


def _check_scan(c, dy, dfinal, worst):
    final, saved = torch.empty_like(c["state"]), sc.selective_scan_saved(c["x"], c["A"])
    y = sc.selective_scan(**c, final_state=final, saved=saved)
    g = sc.selective_scan_grad(dy, **c, saved=saved, dfinal_state=dfinal)
    names = {"x": "dx", "dt": "ddt", "A": "dA", "B": "dB", "C": "dC", "D": "dD", "z": "dz", "dt_bias": "ddt_bias",
             "state": "dstate"}
    batch, length, channels = c["x"].shape
    states, dtype = c["A"].shape[1], c["x"].dtype
    with torch.device("cuda"):
        r = ref.scan(**c, dy=dy, dfinal=dfinal)
    _near("y", y, r["y"])
    _near("final", final, r["final"])
    for k, v in g.items():
        _near("d" + k, v, r[names[k]])
    if not worst:
        return
    with torch.device("cuda"):
        m = ref.scan(**c, dy=dy, dfinal=dfinal, sizes=True)
        # dz = dy y0 sig (1 + z (1 - sig)), whose terms cancel near z = -1.28
        plain = ref.scan(**{k: v for k, v in c.items() if k != "z"}, sizes=True)["y"]
    z = c["z"].double()
    m["dz"] = dy.double().abs() * plain * torch.sigmoid(z) * (1 + z.abs() * torch.sigmoid(-z))
    ref.check("y", y, r["y"], m["y"], dtype, length, states + 1)
    terms = {"A": batch * length, "D": batch * length, "dt_bias": batch * length, "B": channels, "C": channels}
    for k, v in g.items():
        ref.check("d" + k, v, r[names[k]], m[names[k]], v.dtype, length, terms.get(k, states + 1))


@pytest.mark.parametrize("dtype,packed", [(torch.float32, False), (torch.float32, True), (torch.bfloat16, True)])
@pytest.mark.parametrize("batch,length,channels,states,groups,chunk_tiles,run_tiles", [
    (8, 1024, 1024, 16, 1, 16, 16),   # whole tiles, a run a chunk
    (16, 640, 1000, 16, 1, 20, 10),   # two runs a chunk
    (12, 1000, 1024, 16, 1, 21, 21),  # the last tile is half full
    (8, 1000, 513, 16, 1, 9, 9),      # rows off the 16-byte path
    (24, 500, 1026, 16, 2, 32, 32),   # one chunk
])
def test_scan(batch, length, channels, states, groups, chunk_tiles, run_tiles, dtype, packed):
    tiles = -(-length // sc.SC_SSM_SAVE)
    chunks, runs = _scan_plan(batch, length, channels, states, groups)
    assert (-(-tiles // chunks), -(-tiles // runs)) == (chunk_tiles, run_tiles)
    _check_scan(*_scan_case(batch, length, channels, states, groups, dtype, packed), worst=dtype == torch.float32)


@pytest.mark.parametrize("batch,length,channels,states,groups", [
    (8, 900, 1280, 24, 1), (6, 900, 1540, 6, 2), (4, 1100, 1024, 64, 1), (3, 650, 700, 40, 2)])
def test_scan_of_other_numbers_of_states(batch, length, channels, states, groups):
    tiles = -(-length // sc.SC_SSM_SAVE)
    chunks, runs = _scan_plan(batch, length, channels, states, groups)
    assert chunks > 1 and -(-tiles // chunks) > 8  # the sums of dA are flushed and taken up again
    _check_scan(*_scan_case(batch, length, channels, states, groups, torch.float32, True), worst=False)


def test_scan_gradient_of_the_rates_over_a_long_row():
    """Steps between 0.001 and 0.1, rates 1 to 16, 4096 tokens: 1.4e-6 off if the decays'
    exponentials kept their mean error or dA were one running sum, 0.6e-6 as it is."""
    gen = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * scale

    length, channels, states = 4096, 512, 16
    step = torch.exp(torch.rand(channels, generator=gen, device="cuda") * 4.6052 - 6.9078)
    c = {"x": normal(1, length, channels, scale=0.5), "dt": normal(1, length, channels, scale=0.3),
         "A": -torch.arange(1, states + 1, device="cuda").float() * (0.9 + 0.2 * torch.rand(channels, states, generator=gen, device="cuda")),
         "B": normal(1, length, 1, states), "C": normal(1, length, 1, states), "D": 1 + normal(channels, scale=0.1),
         "z": normal(1, length, channels), "dt_bias": step + torch.log(-torch.expm1(-step))}
    dy, saved = normal(1, length, channels, scale=0.01), sc.selective_scan_saved(c["x"], c["A"])
    sc.selective_scan(**c, saved=saved)
    got = sc.selective_scan_grad(dy, **c, saved=saved)["A"]
    with torch.device("cuda"):
        want = ref.scan(**c, dy=dy)["dA"]
    _near("dA", got, want, 1e-6)


@pytest.mark.parametrize("length,channels,states", [(333, 20, 5), (1000, 8, 32), (4000, 64, 16)])
def test_short_chunks(length, channels, states):
    """Few channels: chunks of few tiles, forward and back, and many joins."""
    assert sc.load().sc_selective_scan_workspace_bytes(1, length, channels, states, 1) > 0
    for packed in (False, True):
        _check_scan(*_scan_case(1, length, channels, states, 1, torch.float32, packed), worst=False)


# -------------------------------------------------------------- convolution
def _convolution(x, w, b, heads, state, dy):
    """ref.conv in float64 with the tokens side by side."""
    x, w, dy = x.double(), w.double(), dy.double()
    batch, length, channels = x.shape
    width = w.shape[1]
    before = x.new_zeros(batch, width - 1, channels) if state is None else state.double()
    segment = torch.zeros(batch, length, dtype=torch.long, device="cuda") if heads is None else heads.long().cumsum(1)
    line, of = torch.cat([before, x], 1), torch.cat([segment.new_zeros(batch, width - 1), segment], 1)
    sees = [(of[:, k:k + length] == segment).double()[..., None] for k in range(width)]
    pre, size = b.double().expand_as(x).clone(), b.double().abs().expand_as(x).clone()
    for k in range(width):
        term = w[:, k] * line[:, k:k + length] * sees[k]
        pre += term
        size += term.abs()
    dpre = dy * ref.dsilu(pre)
    dsize = dy.abs() * (ref.dsilu(pre).abs() + size)
    dline, dline_size, dw = torch.zeros_like(line), torch.zeros_like(line), torch.zeros_like(w)
    for k in range(width):
        dline[:, k:k + length] += w[:, k] * dpre * sees[k]
        dline_size[:, k:k + length] += w[:, k].abs() * dsize * sees[k]
        dw[:, k] = (dpre * line[:, k:k + length] * sees[k]).sum((0, 1))
    last = line[:, length:] * (of[:, length:] == segment[:, -1:]).double()[..., None]
    return {"y": ref.silu(pre), "size": size, "final": last, "dx": dline[:, width - 1:], "dx_size": dline_size[:, width - 1:],
            "dstate": dline[:, :width - 1], "dweight": dw, "dbias": dpre.sum((0, 1))}


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("batch,length,channels,width,run", [
    (8, 1280, 4096, 4, 256), (4, 1300, 4096, 8, 128), (8, 700, 2048, 8, 64), (3, 2100, 2050, 8, 64),
    (2, 3000, 4099, 4, 128), (2, 2500, 1024, 4, 32), (1, 5000, 1000, 5, 32), (1, 1300, 2048, 7, 16)])
def test_convolution(batch, length, channels, width, run, dtype, packed):
    scratch = sc.load().sc_causal_conv_grad_workspace_bytes(batch, length, channels, width) - WORKSPACE_HEAD
    assert scratch == batch * -(-length // run) * (width + 1) * channels * 4
    gen = torch.Generator(device="cuda").manual_seed(length + channels)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").to(dtype)

    x, w, b, dy = normal(batch, length, channels), normal(channels, width), normal(channels), normal(batch, length, channels)
    heads = torch.rand(batch, length, generator=gen, device="cuda") < 0.02 if packed else None
    state = normal(batch, width - 1, channels) if packed else None
    final = torch.empty(batch, width - 1, channels, dtype=dtype, device="cuda")
    y = sc.causal_conv(x, w, b, heads=heads, state=state, final_state=final)
    g = sc.causal_conv_grad(dy, x, w, b, heads=heads, state=state)
    r = _convolution(x, w, b, heads, state, dy)
    assert torch.equal(final, r["final"].to(dtype))
    # a few roundings an element; sums over tokens in runs of up to 256 and then of runs
    for name, got, want in (("y", y, r["y"]), ("x", g["x"], r["dx"]), ("weight", g["weight"], r["dweight"]),
                            ("bias", g["bias"], r["dbias"])):
        _near(name, got, want, 3e-6)
    ref.check("y", y, r["y"], r["size"] + r["y"].abs(), dtype, 0, width + 1)
    ref.check("dx", g["x"], r["dx"], r["dx_size"], dtype, 0, width + 1)
    if packed:
        _near("state", g["state"], r["dstate"], 3e-6)
