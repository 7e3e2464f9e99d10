"""Gradients through the block operators' own entry points: as torch records them,
against the gradient calls bit by bit, and a block of all of them against differences."""
import pytest
import torch

import block_reference as ref
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
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("wide", [True, False])
def test_layer_norm(wide, residual, dtype):
    kind = torch.float32 if wide else dtype
    x, w, b = _leaf(_normal(3, 5, 72, dtype=dtype)), _leaf(_normal(72, dtype=kind)), _leaf(_normal(72, seed=1, dtype=kind))
    r = _leaf(_normal(3, 5, 72, seed=2, dtype=dtype)) if residual else None
    dy, ds = _normal(3, 5, 72, seed=3, dtype=dtype), _normal(3, 5, 72, seed=4, dtype=dtype)
    out = sc.layer_norm(x, w, b, residual=r)
    (torch.autograd.backward(out, (dy, ds)) if residual else out.backward(dy))
    with torch.no_grad():
        saved = sc.layer_norm_saved(x)
        y = sc.layer_norm(x, w, b, residual=r, saved=saved)
        s = y[1] if residual else x
        want = sc.layer_norm_grad(dy, s, w, b, saved=saved, dsum=ds if residual else None)
    assert torch.equal(out[0] if residual else out, y[0] if residual else y)
    assert torch.equal(x.grad, want["x"])
    if residual:
        assert torch.equal(r.grad, want["x"]) and r.grad.data_ptr() != x.grad.data_ptr()
    assert torch.equal(w.grad, want["weight"].to(kind)) and torch.equal(b.grad, want["bias"].to(kind))


def test_layer_norm_in_part():
    """One result used, one input that asks."""
    x, r, w = _normal(6, 40), _normal(6, 40, seed=1), _normal(40, seed=2)
    a = _leaf(x)
    y, s = sc.layer_norm(a, w, residual=r)
    s.backward(r)
    assert torch.equal(a.grad, r)
    a = _leaf(x)
    y, s = sc.layer_norm(a, w, residual=r)
    y.sum().backward()
    saved = sc.layer_norm_saved(x)
    sc.layer_norm(x, w, residual=r, saved=saved)
    want = sc.layer_norm_grad(torch.ones_like(x), x + r, w, saved=saved)
    assert torch.equal(a.grad, want["x"])
    p = _leaf(w)
    sc.layer_norm(x, p, residual=r)[0].sum().backward()
    assert torch.equal(p.grad, want["weight"])
    assert not sc.layer_norm(x, w).requires_grad
    with pytest.raises(ValueError, match="out"):
        sc.layer_norm(_leaf(x), out=torch.empty_like(x))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("activation", ["sigmoid", None])
@pytest.mark.parametrize("full", [True, False])
def test_gated_scan(full, activation, dtype):
    joint = _leaf(_normal(2, 45, 160, dtype=dtype, scale=0.4))
    state = _leaf(_normal(2, 80)) if full else None
    heads = torch.arange(45, device="cuda").eq(20).expand(2, 45).contiguous() if full else None
    x, g = joint.chunk(2, -1)
    final = torch.empty(2, 80, device="cuda")
    y = sc.gated_scan(x, g, activation, heads, state, final)
    assert not final.requires_grad
    dy = _normal(2, 45, 80, seed=2, dtype=dtype)
    y.backward(dy)
    with torch.no_grad():
        saved = sc.gated_scan_saved(x)
        assert torch.equal(y, sc.gated_scan(x, g, activation, heads, state, saved=saved))
        want = sc.gated_scan_grad(dy, x, g, activation, heads, state, saved)
    assert torch.equal(joint.grad, torch.cat([want["x"], want["gate"]], -1))
    if full:
        assert torch.equal(state.grad, want["state"])
    with pytest.raises(RuntimeError, match="gated_scan_step"):
        sc.gated_scan_step(_leaf(x[:, 0]), g[:, 0].detach(), _normal(2, 80)).sum().backward()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("weighted", [True, False])
def test_experts(weighted, dtype):
    ids = torch.randint(-1, 6, (30, 3), generator=torch.Generator().manual_seed(1)).cuda()
    order = sc.expert_sort(ids, 6)
    x, w = _leaf(_normal(30, 40, dtype=dtype)), _leaf(_normal(30, 3, seed=1).abs()) if weighted else None
    rows = sc.expert_gather(x, order)
    rows.retain_grad()
    out = sc.expert_combine(rows, order, w)
    dout = _normal(30, 40, seed=2, dtype=dtype)
    out.backward(dout)
    with torch.no_grad():
        assert torch.equal(rows, sc.expert_gather(x, order))
        want = sc.expert_combine_grad(dout, rows, order, w)
        assert torch.equal(rows.grad, want["y"])
        assert torch.equal(x.grad, sc.expert_gather_grad(want["y"], order))
        if weighted:
            assert torch.equal(w.grad, want["weights"])


def test_a_captured_step():
    """Forward and backward in one graph, replayed on other inputs (without a norm's
    parameters, whose gradients need scratch memory)."""
    x, g = _leaf(_normal(2, 40, 64)), _leaf(_normal(2, 40, 64, seed=1))
    ids = torch.randint(0, 5, (80, 2), generator=torch.Generator().manual_seed(1)).cuda()
    share, dy = _leaf(_normal(80, 2, seed=2)), _normal(80, 64, seed=3)

    def step():
        y = sc.layer_norm(sc.gated_scan(x, g), residual=x)[0].flatten(0, 1)
        order = sc.expert_sort(ids, 5)
        out = sc.expert_combine(sc.expert_gather(y, order), order, share)
        return out, *torch.autograd.grad(out, (x, g, share), dy)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        made = step()
    with torch.no_grad():
        x.copy_(x.flip(1))
        ids.copy_(ids.flip(0))
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(made, step()))


def _block(p, x, ids, heads, library):
    """Norm, gated recurrence, its way back to the stream, norm, experts (a matrix each),
    and back: by the library, or from the definitions in float64."""
    n_experts, choices = p["up"].shape[0], ids.shape[1]
    if library:
        h = sc.layer_norm(x, p["w1"], p["b1"])
        u, g = (h @ p["in"]).chunk(2, -1)
        y, stream = sc.layer_norm(sc.gated_scan(u, g, heads=heads) @ p["out"], p["w2"], rms=True, residual=x)
        order = sc.expert_sort(ids, n_experts)
        rows = sc.expert_gather(y.flatten(0, 1), order)
        at = order.offsets.tolist()
        made = torch.cat([torch.tanh(rows[at[e]:at[e + 1]] @ p["up"][e]) for e in range(n_experts)] + [rows[at[-1]:]])
        return stream + sc.expert_combine(made, order, p["share"]).view_as(stream)
    c = x - x.mean(-1, keepdim=True)
    h = c / (c.pow(2).mean(-1, keepdim=True) + 1e-5).sqrt() * p["w1"] + p["b1"]
    u, g = (h @ p["in"]).chunk(2, -1)
    state, ys = torch.zeros_like(u[:, 0]), []
    for t in range(x.shape[1]):
        f = torch.sigmoid(g[:, t])
        state = f * (state * (~heads[:, t, None])) + (1 - f) * u[:, t]
        ys.append(state)
    stream = x + torch.stack(ys, 1) @ p["out"]
    y = (stream / (stream.pow(2).mean(-1, keepdim=True) + 1e-5).sqrt() * p["w2"]).flatten(0, 1)
    out = torch.zeros_like(y)
    for j in range(choices):
        for t in range(len(y)):
            if ids[t, j] >= 0:
                out[t] = out[t] + p["share"][t, j] * torch.tanh(y[t] @ p["up"][ids[t, j]])
    return stream + out.view_as(stream)


def test_a_block_of_them_together():
    """Outputs and gradients of the run as a model has it, against float64 torch over the
    same formulas, and the gradients' product with a direction against a difference."""
    gen = torch.Generator().manual_seed(3)
    dim, batch, length = 24, 2, 21
    p = {"w1": 1 + 0.1 * torch.randn(dim, generator=gen), "b1": 0.1 * torch.randn(dim, generator=gen),
         "in": torch.randn(dim, 2 * dim, generator=gen) / dim ** 0.5, "out": torch.randn(dim, dim, generator=gen) / dim ** 0.5,
         "w2": 1 + 0.1 * torch.randn(dim, generator=gen), "up": torch.randn(4, dim, dim, generator=gen) / dim ** 0.5,
         "share": torch.rand(batch * length, 2, generator=gen)}
    x, dy = torch.randn(batch, length, dim, generator=gen), torch.randn(batch, length, dim, generator=gen)
    ids = torch.randint(-1, 4, (batch * length, 2), generator=gen)
    heads = torch.rand(batch, length, generator=gen) < 0.15
    exact = {k: v.double().requires_grad_() for k, v in (p | {"x": x}).items()}
    want = _block(exact, exact["x"], ids, heads, False)
    want.backward(dy.double())
    mine = {k: v.cuda().requires_grad_() for k, v in (p | {"x": x}).items()}
    torch.backends.cuda.matmul.allow_tf32 = False
    got = _block(mine, mine["x"], ids.cuda(), heads.cuda(), True)
    got.backward(dy.cuda())
    # Each of some ten steps (norms, products over 24, a recurrence of 21 tokens) adds at most 40 x 2^-24 of its
    # values' size to a result of O(1) to O(10) and passes earlier errors on with factors of O(1) to O(5):
    # 1e-4 of the largest value is ten times that, and a wrong term would be of the size of the values.
    for name, a, b in [("out", got, want)] + [(k, mine[k].grad, exact[k].grad) for k in exact]:
        assert (a.detach().double().cpu() - b.detach()).abs().max() <= 1e-4 * b.detach().abs().max(), name
    direction = {k: torch.randn(v.shape, generator=gen).double() for k, v in exact.items()}

    def at(step):
        q = {k: (v + step * direction[k]).detach() for k, v in exact.items()}
        return (_block(q, q["x"], ids, heads, False) * dy).sum().item()

    slope = (at(1e-5) - at(-1e-5)) / 2e-5
    along = sum((mine[k].grad.double().cpu() * direction[k]).sum().item() for k in exact)
    size = sum((mine[k].grad.double().cpu() * direction[k]).abs().sum().item() for k in exact)
    assert abs(along - slope) <= 1e-4 * size
