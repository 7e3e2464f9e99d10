"""Gradients through the sequence operators' own entry points: as torch records them,
against the gradient calls bit by bit, and against differences."""
import pytest
import torch

import seq_reference as ref
import stream_compaction_gb300 as sc
from gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def _normal(*shape, seed=0, dtype=torch.float32, scale=1.0):
    gen = torch.Generator().manual_seed(seed + sum(shape))
    return (torch.randn(*shape, generator=gen) * scale).to(dtype).cuda()


def _leaf(t):
    return None if t is None else t.clone().requires_grad_()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_embed(dtype):
    ids = torch.tensor([[3, 0, 9], [-1, 3, 12]], device="cuda")
    weight, dy = _leaf(_normal(12, 20, dtype=dtype)), _normal(2, 3, 20, seed=1, dtype=dtype)
    y = sc.embed(ids, weight, 1.5)
    assert y.requires_grad
    with torch.no_grad():
        assert torch.equal(y, sc.embed(ids, weight, 1.5))
    y.backward(dy)
    assert torch.equal(weight.grad, sc.embed_grad(ids, dy, 12, 1.5))
    assert weight.grad.dtype == dtype and (weight.grad[0] != 0).any() and (weight.grad[1] == 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("activation", ["silu", None])
@pytest.mark.parametrize("full", [True, False])
def test_causal_conv(full, activation, dtype):
    joint = _leaf(_normal(2, 21, 80, dtype=dtype))
    weight, bias = _leaf(_normal(40, 4, dtype=dtype)), _leaf(_normal(40, dtype=dtype)) if full else None
    state = _leaf(_normal(2, 3, 40, dtype=dtype)) if full else None
    heads = torch.arange(21, device="cuda").eq(9).expand(2, 21).contiguous() if full else None
    x, final = joint[:, :, 40:], torch.empty(2, 3, 40, dtype=dtype, device="cuda")
    y = sc.causal_conv(x, weight, bias, activation, heads=heads, state=state, final_state=final)
    assert not final.requires_grad
    dy = _normal(2, 21, 40, seed=2, dtype=dtype)
    y.backward(dy)
    with torch.no_grad():
        again = torch.empty_like(final)
        assert torch.equal(y, sc.causal_conv(x, weight, bias, activation, heads=heads, state=state, final_state=again))
        assert torch.equal(final, again)
        want = sc.causal_conv_grad(dy, x, weight, bias, activation, heads=heads, state=state)
    assert torch.equal(joint.grad[:, :, 40:], want["x"]) and (joint.grad[:, :, :40] == 0).all()
    assert torch.equal(weight.grad, want["weight"].to(dtype))
    if full:
        assert torch.equal(bias.grad, want["bias"].to(dtype)) and torch.equal(state.grad, want["state"])


def _scan_inputs(dtype, full):
    c = {"x": _normal(2, 37, 40, dtype=dtype), "dt": _normal(2, 37, 40, seed=1, dtype=dtype, scale=0.3),
         "A": -0.1 - _normal(40, 16, seed=2).abs(), "B": _normal(2, 37, 2, 16, seed=3, dtype=dtype),
         "C": _normal(2, 37, 2, 16, seed=4, dtype=dtype)}
    if full:
        c |= {"D": _normal(40, seed=5), "z": _normal(2, 37, 40, seed=6, dtype=dtype), "dt_bias": _normal(40, seed=7) - 2,
              "state": _normal(2, 40, 16, seed=8)}
    return {k: _leaf(v) for k, v in c.items()}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("full", [True, False])
def test_selective_scan(full, dtype):
    c = _scan_inputs(dtype, full)
    heads = {"heads": torch.arange(37, device="cuda").eq(20).expand(2, 37).contiguous()} if full else {}
    y = sc.selective_scan(**c, **heads)
    dy = _normal(2, 37, 40, seed=9, dtype=dtype)
    y.backward(dy)
    with torch.no_grad():
        saved = sc.selective_scan_saved(c["x"], c["A"])
        assert torch.equal(y, sc.selective_scan(**c, **heads, saved=saved))
        want = sc.selective_scan_grad(dy, **c, **heads, saved=saved)
    assert set(want) == set(c)
    for k in c:
        assert torch.equal(c[k].grad, want[k]), k


def test_only_what_asks_for_a_gradient_gets_one():
    c = {k: v.detach() for k, v in _scan_inputs(torch.float32, True).items()}
    c["A"].requires_grad_()
    y = sc.selective_scan(**c)
    y.sum().backward()  # the gradient comes in expanded from one number
    assert c["A"].grad is not None and all(v.grad is None for k, v in c.items() if k != "A")
    saved = sc.selective_scan_saved(c["x"], c["A"])
    with torch.no_grad():
        sc.selective_scan(**c, saved=saved)
        assert torch.equal(c["A"].grad, sc.selective_scan_grad(torch.ones_like(y), **c, saved=saved)["A"])
        assert not sc.selective_scan(**c).requires_grad
    assert not sc.selective_scan(**{k: v.detach() for k, v in c.items()}).requires_grad


def test_a_chain_against_differences():
    """embed -> conv -> scan, as torch chains them, along a direction of all parameters:
    against a central difference of the float64 definitions."""
    ids = torch.tensor([[1, 5, 2, 5, 0, 7, 3, 1, 1, 6, 2, 4]])
    p = {"weight": _normal(8, 24, seed=1), "conv": _normal(24, 4, seed=2, scale=0.5), "bias": _normal(24, seed=3),
         "A": -0.1 - _normal(24, 16, seed=4).abs(), "D": _normal(24, seed=5), "dt_bias": _normal(24, seed=6) - 1,
         "B": _normal(1, 12, 1, 16, seed=7), "C": _normal(1, 12, 1, 16, seed=8), "dt": _normal(1, 12, 24, seed=9)}
    dy = _normal(1, 12, 24, seed=10)

    def exact(q):
        u = ref.conv(ref.embed(ids, q["weight"], 1.0), q["conv"], q["bias"])["y"]
        return (ref.scan(u, q["dt"], q["A"], q["B"], q["C"], q["D"], None, q["dt_bias"])["y"] * dy.cpu().double()).sum()

    leaves = {k: _leaf(v) for k, v in p.items()}
    u = sc.causal_conv(sc.embed(ids.cuda(), leaves["weight"]), leaves["conv"], leaves["bias"])
    y = sc.selective_scan(u, leaves["dt"], leaves["A"], leaves["B"], leaves["C"], leaves["D"],
                          dt_bias=leaves["dt_bias"])
    y.backward(dy)
    cpu = {k: v.cpu().double() for k, v in p.items()}
    for name in p:
        along = _normal(*p[name].shape, seed=11).cpu().double()
        step = 1e-5
        slope = (exact({**cpu, name: cpu[name] + step * along}) - exact({**cpu, name: cpu[name] - step * along})) / (2 * step)
        terms = leaves[name].grad.cpu().double() * along
        # truncation: step^2 times third derivatives of O(100) sums; float32 errors: 12 tokens' worth of 2^-24
        assert abs(terms.sum() - slope) <= 1e-4 * terms.abs().sum() + 1e-6, (name, terms.sum(), slope)


def test_on_another_stream():
    c = _scan_inputs(torch.float32, True)
    dy = _normal(2, 37, 40, seed=9)
    sc.selective_scan(**c).backward(dy)
    want = {k: v.grad.clone() for k, v in c.items()}
    for v in c.values():
        v.grad = None
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = sc.selective_scan(**c, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    y.backward(dy)
    torch.cuda.synchronize()
    assert all(torch.equal(c[k].grad, want[k]) for k in c)
    assert sc.sc_release_stream(s.cuda_stream) == sc.SC_OK


def test_refusals():
    weight = _leaf(_normal(12, 20))
    ids = torch.zeros(3, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        sc.embed(ids, weight, out=torch.empty(3, 20, device="cuda"))
    x, w = _leaf(_normal(2, 5, 8)), _normal(8, 4)
    with pytest.raises(ValueError):
        sc.causal_conv(x, w, out=torch.empty(2, 5, 8, device="cuda"))
    with torch.no_grad():
        sc.causal_conv(x, w, out=torch.empty(2, 5, 8, device="cuda"))
    with pytest.raises(ValueError):  # the calls' own checks
        sc.causal_conv(x, w.half())
    # second derivatives are not recorded, and say so
    (g,) = torch.autograd.grad(sc.causal_conv(x, w).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_a_state_overwritten_before_the_gradient_is_noticed():
    x, w = _leaf(_normal(2, 5, 8)), _normal(8, 4)
    a, b = _normal(2, 3, 8, seed=1), torch.empty(2, 3, 8, device="cuda")
    first = sc.causal_conv(x, w, state=a, final_state=b)
    second = sc.causal_conv(x, w, state=b, final_state=a)  # a was the first call's input
    second.sum().backward()
    with pytest.raises(RuntimeError):
        first.sum().backward()


def test_single_tokens_have_no_gradient_and_say_so():
    x, w = _normal(2, 8), _leaf(_normal(8, 4))
    pool, other = torch.zeros(2, 3, 8, device="cuda"), torch.zeros(2, 3, 8, device="cuda")
    y = sc.causal_conv_step(x, pool, w)
    with torch.no_grad():
        assert torch.equal(y, sc.causal_conv_step(x, other, w)) and torch.equal(pool, other)
    assert (pool[:, 2] == x).all()
    with pytest.raises(RuntimeError, match="causal_conv"):
        y.sum().backward()
    A = _leaf(-torch.ones(8, 16, device="cuda"))
    bc, states = _normal(2, 1, 16), torch.zeros(2, 8, 16, device="cuda")
    y = sc.selective_scan_step(x, x, A, bc, bc, states)
    assert (states != 0).any()
    with pytest.raises(RuntimeError, match="selective_scan"):
        y.sum().backward()
