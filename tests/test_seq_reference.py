"""The float64 references of the sequence operators against differences: every
gradient formula against central differences of the forward definition."""
import pytest
import torch

import seq_reference as ref


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _differences(f, tensors, weights, step=1e-5):
    """Gradient of sum(weights * f()) by every element of each tensor, by central differences."""
    grads = []
    for t in tensors:
        g = torch.zeros_like(t)
        flat, out = t.view(-1), g.view(-1)
        for i in range(flat.numel()):
            keep = flat[i].item()
            flat[i] = keep + step
            up = sum((w * o).sum() for w, o in zip(weights, f()))
            flat[i] = keep - step
            down = sum((w * o).sum() for w, o in zip(weights, f()))
            flat[i] = keep
            out[i] = (up - down) / (2 * step)
        grads.append(g)
    return grads


def _close(a, b):
    # central differences in float64: truncation step^2 * f''' and rounding 1e-16 / step, both below 1e-8 of O(1) values
    assert torch.allclose(a, b, rtol=1e-6, atol=1e-7), (a - b).abs().max()


@pytest.mark.parametrize("act", [True, False])
@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("width", [1, 2, 4])
def test_conv_gradients(width, packed, act):
    gen = _gen(width)
    x, dy = (torch.randn(2, 7, 3, generator=gen, dtype=torch.float64) for _ in range(2))
    w, b = torch.randn(3, width, generator=gen, dtype=torch.float64), torch.randn(3, generator=gen, dtype=torch.float64)
    state = torch.randn(2, width - 1, 3, generator=gen, dtype=torch.float64)
    heads = torch.rand(2, 7, generator=gen) < 0.3 if packed else None
    r = ref.conv(x, w, b, heads, state, act, dy)
    dx, dw, db, ds = _differences(lambda: [ref.conv(x, w, b, heads, state, act)["y"]], [x, w, b, state], [dy])
    for got, want in ((r["dx"], dx), (r["dweight"], dw), (r["dbias"], db), (r["dstate"], ds)):
        _close(got, want)


@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("groups,gated", [(1, True), (2, True), (2, False)])
def test_scan_gradients(groups, gated, packed):
    gen = _gen(groups)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, dtype=torch.float64)

    x, dt, dy = normal(2, 5, 4), normal(2, 5, 4), normal(2, 5, 4)
    A, D, bias = -torch.rand(4, 3, generator=gen, dtype=torch.float64) - 0.1, normal(4), normal(4)
    B, C, state, dfinal = normal(2, 5, groups, 3), normal(2, 5, groups, 3), normal(2, 4, 3), normal(2, 4, 3)
    z = normal(2, 5, 4) if gated else None
    heads = torch.rand(2, 5, generator=gen) < 0.3 if packed else None

    def forward():
        r = ref.scan(x, dt, A, B, C, D, z, bias, True, heads, state)
        return [r["y"], r["final"]]

    r = ref.scan(x, dt, A, B, C, D, z, bias, True, heads, state, dy, dfinal)
    names = ["dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dstate"] + (["dz"] if gated else [])
    tensors = [x, dt, A, B, C, D, bias, state] + ([z] if gated else [])
    for name, want in zip(names, _differences(forward, tensors, [dy, dfinal])):
        _close(r[name], want)
