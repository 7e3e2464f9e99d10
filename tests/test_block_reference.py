"""The float64 definitions of the norm, the gated recurrence and the experts' sums
against differences, and a mistake planted in each that its bound has to show."""
import pytest
import torch

import block_reference as ref


def _normal(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed + sum(shape)), dtype=torch.float64)


def _slope(f, tensors, step=1e-6):
    """Derivatives of the number f() by every element of each tensor, by central differences."""
    out = []
    for t in tensors:
        g = torch.zeros_like(t)
        for i in range(t.numel()):
            keep = t.view(-1)[i].item()
            t.view(-1)[i] = keep + step
            up = f()
            t.view(-1)[i] = keep - step
            down = f()
            t.view(-1)[i] = keep
            g.view(-1)[i] = (up - down) / (2 * step)
        out.append(g)
    return out


def _close(a, b):
    # truncation step^2 f''' / 6 and rounding 1e-16 / step of O(1) values
    assert torch.allclose(a, b, rtol=1e-6, atol=1e-7), (a - b).abs().max()


@pytest.mark.parametrize("rms", [True, False])
def test_norm(rms):
    x, w, b = _normal(3, 7), _normal(7, seed=1), _normal(7, seed=2)
    dy, dsum = _normal(3, 7, seed=3), _normal(3, 7, seed=4)

    def f():
        r = ref.norm(x, w, b, 0.1, rms)
        return ((r["y"][0] * dy).sum() + (r["sum"][0] * dsum).sum()).item()

    r = ref.norm(x, w, b, 0.1, rms, dy=dy, dsum=dsum)
    for name, slope in zip(("dx", "dweight", "dbias"), _slope(f, (x, w, b))):
        _close(r[name][0], slope)


@pytest.mark.parametrize("activation", ["sigmoid", None])
@pytest.mark.parametrize("packed", [True, False])
def test_gated(packed, activation):
    x, g, state = _normal(2, 6, 3), _normal(2, 6, 3, seed=1), _normal(2, 3, seed=2)
    heads = torch.tensor([[0, 0, 1, 0, 0, 0], [1, 0, 0, 0, 1, 1]]) if packed else None
    dy, dfinal = _normal(2, 6, 3, seed=3), _normal(2, 3, seed=4)

    def f():
        r = ref.gated(x, g, activation, heads, state)
        return ((r["y"][0] * dy).sum() + (r["final"][0] * dfinal).sum()).item()

    r = ref.gated(x, g, activation, heads, state, dy, dfinal)
    for name, slope in zip(("dx", "dgate", "dstate"), _slope(f, (x, g, state))):
        _close(r[name][0], slope)


def test_experts():
    ids = torch.tensor([[2, 0], [0, -1], [1, 2], [5, 0]])
    offsets, order, place = ref.expert_sort(ids, 3)
    assert offsets == [0, 3, 4, 6] and order == [1, 2, 7, 4, 0, 5, 3, 6] and place == [4, 0, 1, 6, 3, 5, 7, 2]
    y, w, dout = _normal(8, 3), _normal(4, 2, seed=1), _normal(4, 3, seed=2)
    f = lambda: (ref.expert_combine(y, place, 6, 4, 2, w)["out"][0] * dout).sum().item()  # noqa: E731
    r = ref.expert_combine(y, place, 6, 4, 2, w, dout)
    for name, slope in zip(("dy", "dweights"), _slope(f, (y, w))):
        _close(r[name][0], slope)


def _caught(got, pair):
    with pytest.raises(AssertionError):
        ref.check("planted", got, pair)


def test_the_bounds_show_planted_mistakes():
    x, w, b, dy = (_normal(*s, seed=i).float() for i, s in enumerate([(5, 200), (200,), (200,), (5, 200)]))
    r = ref.norm(x, w, b, dy=dy)
    for k in ("y", "dx", "dweight"):
        ref.check(k, r[k][0].float(), r[k])
    _caught(ref.norm(x, w, b, 1e-4)["y"][0].float(), r["y"])               # another eps
    _caught((ref.norm(x, w, b, rms=True)["y"][0]).float(), r["y"])         # no mean
    short = ref.norm(x[:, :-1], w[:-1], b[:-1])["y"][0].float()            # a sum without its last element
    _caught(short, (r["y"][0][:, :-1], r["y"][1][:, :-1]))
    _caught(ref.norm(x[:-1], w, b, dy=dy[:-1])["dweight"][0].float(), r["dweight"])  # a row left out
    x, g, dy = _normal(1, 40, 8).float(), _normal(1, 40, 8, seed=1).float(), _normal(1, 40, 8, seed=2).float()
    state = _normal(1, 8, seed=3).float()
    heads = torch.zeros(1, 40).index_fill_(1, torch.tensor([20]), 1)
    r = ref.gated(x, g, "sigmoid", heads, state, dy)
    for k in ("y", "dx", "dgate", "dstate"):
        ref.check(k, r[k][0].float(), r[k])
    other = ref.gated(x, g, "sigmoid", heads.roll(1, 1), state, dy)       # a segment one token late
    for k in ("y", "dx", "dgate"):
        _caught(other[k][0].float(), r[k])
    _caught(ref.gated(x, g, "sigmoid", heads, None, dy)["y"][0].float(), r["y"])
