"""The gated recurrence, its gradient and its form for one token against float64."""
import pytest
import torch

import block_reference as ref
import stream_compaction_gb300 as sc
from gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def _normal(*shape, seed=0, dtype=torch.float32, scale=1.0):
    gen = torch.Generator().manual_seed(seed + sum(shape))
    return (torch.randn(*shape, generator=gen) * scale).to(dtype)


def _case(batch, length, channels, dtype, activation="sigmoid", packed=False, often=0.1):
    """Gates of channels that remember one token to thousands."""
    x, dy = _normal(batch, length, channels, dtype=dtype), _normal(batch, length, channels, seed=1, dtype=dtype)
    g = _normal(batch, length, channels, seed=2) + torch.linspace(-4, 8, channels)
    g = torch.sigmoid(g) * torch.where(torch.arange(channels) % 5 == 0, -1.0, 1.0) if activation is None else g.clamp(-12, 12)
    gen = torch.Generator().manual_seed(length)
    heads = torch.rand(batch, length, generator=gen) < often if packed else None
    state = _normal(batch, channels, seed=3) if packed else None
    return x, g.to(dtype), heads, state, dy


def _run(x, g, heads, state, dy, activation, dfinal=None):
    x, g, heads, state, dy, dfinal = (None if t is None else t.cuda() for t in (x, g, heads, state, dy, dfinal))
    final = torch.full((x.shape[0], x.shape[2]), -7.0, device="cuda")
    saved = sc.gated_scan_saved(x)
    y = sc.gated_scan(x, g, activation, heads, state, final, saved)
    grads = sc.gated_scan_grad(dy, x, g, activation, heads, state, saved, dfinal)
    assert set(grads) == {"x", "gate"} | ({"state"} if state is not None else set())
    return y, final, grads


def _check(case, activation, got, dfinal=None):
    r = ref.gated(case[0], case[1], activation, case[2], case[3], case[4], dfinal)
    y, final, grads = got
    ref.check("y", y, r["y"])
    ref.check("final", final, r["final"])
    ref.check("dx", grads["x"], r["dx"])
    ref.check("dgate", grads["gate"], r["dgate"])
    if "state" in grads:
        ref.check("dstate", grads["state"], r["dstate"])


# tiles of 16 tokens; 1, 4 or 8 of them a CTA; up to 8 CTAs a cluster
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("activation", ["sigmoid", None])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("batch,length,channels", [
    (1, 1, 1), (2, 2, 64), (3, 15, 33), (1, 16, 32), (2, 17, 65), (1, 64, 31), (2, 65, 130), (1, 128, 2), (3, 129, 66),
    (1, 300, 100), (2, 1025, 40), (1, 2500, 70), (12, 1100, 40)])
def test_forward_and_gradient(batch, length, channels, packed, activation, dtype):
    case = _case(batch, length, channels, dtype, activation, packed)
    dfinal = _normal(batch, channels, seed=9) if packed else None
    got = _run(*case, activation, dfinal)
    _check(case, activation, got, dfinal)
    again = _run(*case, activation, dfinal)
    assert torch.equal(got[0], again[0]) and all(torch.equal(got[2][k], again[2][k]) for k in got[2])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("batch,channels", [(40, 300), (3, 6000)])
def test_more_rows_than_the_machine_holds(batch, channels, dtype):
    """Single CTAs and small clusters in place of clusters of 8."""
    case = _case(batch, 150, channels, dtype, packed=True, often=0.02)
    _check(case, "sigmoid", _run(*case, "sigmoid"))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset,channels", [(0, 64), (1, 64), (64, 64), (3, 37), (2, 66)])
def test_slices_of_a_joint_buffer(offset, channels, dtype):
    """x and gate as columns of wider rows, aligned or not; y into such columns."""
    joint = torch.cat([_normal(2, 50, 140, dtype=dtype), _normal(2, 50, 140, seed=1, dtype=dtype)], -1).cuda()
    x, g = joint[:, :, offset:offset + channels], joint[:, :, 140 + offset:140 + offset + channels]
    wide = _normal(2, 50, 150, seed=2, dtype=dtype).cuda()
    dy = wide[:, :, offset:offset + channels]
    out = torch.full((2, 50, 141), -7.0, dtype=dtype, device="cuda")
    saved = sc.gated_scan_saved(x)
    y = sc.gated_scan(x, g, saved=saved, out=out[:, :, offset:offset + channels])
    assert (out[:, :, :offset] == -7).all() and (out[:, :, offset + channels:] == -7).all()
    r = ref.gated(x.cpu(), g.cpu(), dy=dy.cpu())
    ref.check("y", y, r["y"])
    grads = sc.gated_scan_grad(dy, x, g, saved=saved)
    ref.check("dx", grads["x"], r["dx"])
    ref.check("dgate", grads["gate"], r["dgate"])


@pytest.mark.parametrize("dtype", DTYPES)
def test_layouts(dtype):
    """Tokens before rows, rows with gaps between them, one row for all."""
    case = _case(3, 70, 64, dtype)
    r = ref.gated(case[0], case[1], dy=case[4])
    gap = torch.zeros(3, 70 * 64 + 24, dtype=dtype, device="cuda")

    def turned(t):
        return t.transpose(0, 1).contiguous().transpose(0, 1)

    def apart(t):
        v = gap.clone()[:, :70 * 64].view(3, 70, 64)
        v.copy_(t)
        return v

    for lay in (turned, apart):
        x, g, dy = (lay(case[i].cuda()) for i in (0, 1, 4))
        assert not x.is_contiguous()
        out, saved = lay(torch.zeros_like(x)), sc.gated_scan_saved(x)
        ref.check("y", sc.gated_scan(x, g, saved=saved, out=out), r["y"])
        grads = sc.gated_scan_grad(dy, x, g, saved=saved)
        ref.check("dx", grads["x"], r["dx"])
        ref.check("dgate", grads["gate"], r["dgate"])
    x, g = case[0][:1].cuda().expand(3, 70, 64), case[1][:1].cuda().expand(3, 70, 64)
    ref.check("one row", sc.gated_scan(x, g), [v[:1].expand(3, 70, 64) for v in r["y"]])


def test_more_than_2_31_elements():
    """Offsets beyond 32 bits: the last channels of the last row as a call of their own has them."""
    shape, dtype = (2, 270000, 4096), torch.bfloat16
    x = torch.randn(shape, dtype=dtype, device="cuda")
    g = torch.randn(shape, dtype=dtype, device="cuda")
    saved = sc.gated_scan_saved(x)
    y = sc.gated_scan(x, g, saved=saved)
    part = [t[1:, :, -64:].contiguous() for t in (x, g, y)]
    small = sc.gated_scan_saved(part[0])
    want = sc.gated_scan(part[0], part[1], saved=small)
    # other splits of the length: float32 differences far below bfloat16's steps, so neighbours at most
    assert (part[2].float() - want.float()).abs().max() <= 2 ** -7 * want.abs().max()
    grads = sc.gated_scan_grad(y, x, g, saved=saved)
    want = sc.gated_scan_grad(part[2], part[0], part[1], saved=small)
    for k in ("x", "gate"):
        got = grads[k][1:, :, -64:].float()
        assert (got - want[k].float()).abs().max() <= 2 ** -7 * want[k].abs().max(), k


@pytest.mark.parametrize("activation", ["sigmoid", None])
@pytest.mark.parametrize("channels", [64, 33])
def test_prompt_in_parts_and_token_by_token(channels, activation):
    """A row cut anywhere and continued from its state, and single tokens after a prompt."""
    x, g, _, _, dy = _case(3, 70, channels, torch.float32, activation)
    r = ref.gated(x, g, activation)
    x, g = x.cuda(), g.cuda()
    for cut in (1, 16, 40, 69):
        mid, end = (torch.empty(3, channels, device="cuda") for _ in range(2))
        first = sc.gated_scan(x[:, :cut], g[:, :cut], activation, final_state=mid)
        second = sc.gated_scan(x[:, cut:], g[:, cut:], activation, state=mid, final_state=end)
        ref.check("parts", torch.cat([first, second], 1), r["y"])
        ref.check("end", end, r["final"])
    pool = torch.full((7, channels), 5.0, device="cuda")
    slots = torch.tensor([4, 0, 6], dtype=torch.int32, device="cuda")
    pool[slots.long()] = 0.0
    made = [sc.gated_scan_step(x[:, t], g[:, t], pool, activation, slots) for t in range(70)]
    ref.check("tokens", torch.stack(made, 1), r["y"])
    ref.check("pool", pool[slots.long()], r["final"])
    assert (pool[[1, 2, 3, 5]] == 5).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("batch,channels", [(1, 1), (5, 64), (3, 37), (130, 260)])
def test_one_token(batch, channels, dtype):
    x, g, _, _, _ = _case(batch, 1, channels, dtype)
    pool = _normal(batch + 3, channels, seed=5)
    slots = torch.randperm(batch + 3, generator=torch.Generator().manual_seed(1))[:batch].to(torch.int32)
    slots[0] = batch + 3 if batch % 2 else -1  # sits out
    dev = pool.cuda()
    y = sc.gated_scan_step(x[:, 0].cuda(), g[:, 0].cuda(), dev, slots=slots.cuda())
    r = ref.gated(x, g, state=pool[slots.long().clamp(0, batch + 2)])
    want = r["y"][0][:, 0].clone()
    want[0] = 0
    ref.check("y", y, (want, r["y"][1][:, 0]))
    after, bound = pool.double(), torch.zeros_like(pool).double()
    after[slots[1:].long()] = r["final"][0][1:]
    bound[slots[1:].long()] = r["final"][1][1:]
    ref.check("pool", dev, (after, bound))
    assert torch.equal(dev[bound.cuda().sum(1) == 0], pool.cuda()[bound.cuda().sum(1) == 0])
    own = pool[:batch].cuda()
    y2 = sc.gated_scan_step(x[:, 0].cuda(), g[:, 0].cuda(), own)  # row r in row r
    ref.check("own rows", y2, tuple(v[:, 0] for v in ref.gated(x, g, state=pool[:batch])["y"]))


def test_infinities_stay_behind_the_next_segment():
    """What a segment's start drops is not multiplied by 0; a state that is not finite
    stays so up to there."""
    for channels, activation in ((64, "sigmoid"), (33, None)):
        x, g, _, state, dy = _case(2, 400, channels, torch.float32, activation)
        heads = torch.zeros(2, 400, dtype=torch.bool)
        heads[:, [7, 150, 333]] = True
        state = torch.full((2, channels), float("inf"))
        x[0, 160:170], x[1, 340] = float("nan"), float("-inf")
        got = _run(x, g, heads, state, dy, activation)
        y = got[0].cpu()
        assert not y[:, :7].isfinite().any()
        ok = ref.gated(x.nan_to_num(0, 0, 0), g, activation, heads, state.nan_to_num(0, 0, 0))["y"]
        for rows, a, b in (([0, 1], 7, 150), ([0], 150, 160), ([1], 150, 333), ([0], 333, 400), ([1], 333, 340)):
            for row in rows:
                ref.check("after a start", y[row, a:b], (ok[0][row, a:b], ok[1][row, a:b]))
        assert not y[0, 160:333].isfinite().any() and not y[1, 340:].isfinite().any()


def test_extreme_gates():
    x = torch.ones(1, 40, 64)
    for value, want in ((200.0, 0.0), (-200.0, 1.0), (float("inf"), 0.0), (float("-inf"), 1.0)):
        for dtype in DTYPES:
            y = sc.gated_scan(x.to(dtype).cuda(), torch.full((1, 40, 64), value, dtype=dtype, device="cuda"))
            assert (y == want).all(), (value, dtype)


def test_nothing_to_do():
    z = torch.zeros(2, 0, 8, device="cuda")
    state, final = torch.rand(2, 8, device="cuda"), torch.empty(2, 8, device="cuda")
    assert sc.gated_scan(z, z, state=state, final_state=final).shape == z.shape
    assert torch.equal(final, state)
    g = sc.gated_scan_grad(z, z, z, state=state, saved=sc.gated_scan_saved(z), dfinal_state=state)
    assert torch.equal(g["state"], state)
    for shape in ((0, 5, 8), (2, 5, 0)):
        e = torch.zeros(shape, device="cuda")
        assert sc.gated_scan(e, e).shape == shape


def test_refusals():
    x = torch.zeros(2, 5, 8, device="cuda")
    state, saved = torch.zeros(2, 8, device="cuda"), sc.gated_scan_saved(x)
    for bad in (dict(activation="tanh"), dict(heads=torch.zeros(2, 4, dtype=torch.bool, device="cuda")),
                dict(state=state[:1]), dict(state=state.half()), dict(saved=saved[:1]), dict(out=x.half()),
                dict(heads=torch.zeros(2, 5, device="cuda"))):
        with pytest.raises(ValueError):
            sc.gated_scan(x, x.clone(), **bad)
    for a, b in ((x, x[:, :4]), (x, x.half()), (x[0], x[0]), (x.double(), x.double()), (x.cpu(), x.cpu())):
        with pytest.raises(ValueError):
            sc.gated_scan(a, b)
    with pytest.raises(sc.ScanError):
        sc.gated_scan(x, x.clone(), out=x)
    with pytest.raises(sc.ScanError):
        sc.gated_scan(x, x.clone(), state=state, final_state=state)
    with pytest.raises(ValueError, match="saved"):
        sc.gated_scan_grad(x, x, x)
    with pytest.raises(ValueError):
        sc.gated_scan_step(x[:, 0], x[:, 0], state, slots=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(sc.ScanError):
        sc.gated_scan_step(x[:, 0], x[:, 1], state[:1])


def test_streams_and_graphs():
    """On another stream; forward, gradient and single token captured, replayed on other inputs."""
    x, g, heads, state, dy = (t.cuda() for t in _case(2, 500, 96, torch.bfloat16, packed=True))

    def all_of():
        final, saved = torch.empty_like(state), sc.gated_scan_saved(x)
        y = sc.gated_scan(x, g, "sigmoid", heads, state, final, saved)
        grads = sc.gated_scan_grad(dy, x, g, "sigmoid", heads, state, saved)
        pool = state.clone()
        return [y, final, *grads.values(), sc.gated_scan_step(x[:, 0], g[:, 0], pool), pool]

    want = all_of()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = all_of()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        made = all_of()
    x.copy_(x.flip(1))
    dy.mul_(2)
    want = all_of()
    for _ in range(2):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(made, want))
