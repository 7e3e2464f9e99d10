"""The gated recurrence with decays as they are given, of any size: where the product of a
run of them passes float32's range, states that do not are what the recurrence says.

Bounds: those of block_reference.gated, whose terms are relative to the recurrence over
absolute values and hold for decays of any size."""
import pytest
import torch

import block_reference as ref
import stream_compaction_gb300 as sc
from gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def _run(x, g, heads, state, dy, dfinal):
    x, g, heads, state, dy, dfinal = (None if t is None else t.cuda() for t in (x, g, heads, state, dy, dfinal))
    final, saved = torch.empty(x.shape[0], x.shape[2], device="cuda"), sc.gated_scan_saved(x)
    y = sc.gated_scan(x, g, None, heads, state, final, saved)
    return y, final, sc.gated_scan_grad(dy, x, g, None, heads, state, saved, dfinal)


# CTAs of 4 and of 8 warps; alone, in clusters of 2 to 8 and of 16; rows aligned or not
SHAPES = [(1, 40, 64), (2, 300, 64), (1, 700, 37), (1, 4200, 32), (1, 4100, 33), (40, 80, 1024), (40, 70, 1023), (8, 170, 256)]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("batch,length,channels", SHAPES)
def test_nothing_times_infinity(batch, length, channels, dtype, packed):
    """Zero states and inputs under decays whose products overflow stay zero; channels beside
    them are what they are without."""
    gen = torch.Generator().manual_seed(length)
    x, dy = (torch.randn(batch, length, channels, generator=gen).to(dtype) for _ in range(2))
    g = (torch.rand(batch, length, channels, generator=gen) * 2 - 1).to(dtype)
    state, dfinal = torch.randn(batch, channels, generator=gen), torch.randn(batch, channels, generator=gen)
    heads = torch.rand(batch, length, generator=gen) < 0.02 if packed else None
    plain = _run(x, g, heads, state, dy, dfinal)
    large = torch.arange(channels) % 3 == 1
    g[:, :, large], x[:, :, large], dy[:, :, large], state[:, large], dfinal[:, large] = 1e10, 0, 0, 0, 0
    y, final, grads = _run(x, g, heads, state, dy, dfinal)
    for t in (y, final, grads["x"], grads["gate"], grads["state"]):
        assert (t[..., large] == 0).all()
    for a, b in ((y, plain[0]), (final, plain[1]), *((grads[k], plain[2][k]) for k in grads)):
        assert torch.equal(a[..., ~large], b[..., ~large])


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("batch,length,channels", SHAPES)
def test_products_that_overflow_before_a_state_does(batch, length, channels, packed):
    """Runs of 16 tokens whose decays multiply to 10^64, between others that bring the states
    back: these go from 10^-36 to 10^28 and to 10^-4 and on."""
    period = torch.tensor([1e4] * 16 + [1e-4] * 8 + [1.0] * 8 + [1e-4] * 8 + [1.0] * 8)
    token = torch.arange(length) % 48
    gen = torch.Generator().manual_seed(length)
    spread = 0.5 + torch.rand(batch, length, channels, generator=gen)
    g = period[token][None, :, None].expand(batch, length, channels)
    g = (g * torch.where(torch.rand(batch, length, channels, generator=gen) < 0.3, -1.0, 1.0)).contiguous()
    x = torch.zeros(batch, length, channels)
    state = spread[:, 0] * 1e-36
    heads = torch.rand(batch, length, generator=gen) < 0.01 if packed else None
    dy, dfinal = torch.zeros(batch, length, channels), torch.zeros(batch, channels)
    dy[:, 15::48] = spread[:, 15::48] * 1e-36  # grows to 10^28 on the way back through the run
    r = ref.gated(x, g, None, heads, state, dy, dfinal)
    y, final, grads = _run(x, g, heads, state, dy, dfinal)
    floor = 2.0 ** -126  # below it a value has fewer digits
    for name, got in (("y", y), ("final", final), ("dx", grads["x"]), ("dgate", grads["gate"]), ("dstate", grads["state"])):
        want, bound = r[name]
        ref.check(name, got, (want, bound + floor))
