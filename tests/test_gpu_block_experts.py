"""Tokens sorted by expert, their rows there and back, and the gradients."""
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


def _normal(*shape, seed=0, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed + sum(shape))).to(dtype)


def _ids(tokens, choices, experts, dropped, kind=torch.int64, skew=False):
    gen = torch.Generator().manual_seed(tokens + choices)
    ids = torch.randint(0, experts, (tokens, choices), generator=gen)
    if skew:
        ids = torch.where(torch.rand(tokens, choices, generator=gen) < 0.9, min(3, experts - 1), ids)
    if dropped:
        out = torch.rand(tokens, choices, generator=gen) < dropped
        wrong = torch.tensor([-1, experts, -2 ** 31, 2 ** 31 - 1] if kind == torch.int32 else [-1, experts, -2 ** 62, 2 ** 32])
        ids = torch.where(out, wrong[torch.randint(0, 4, ids.shape, generator=gen)], ids)
    return ids.to(kind)


def _sorted(ids, experts):
    order = sc.expert_sort(ids.cuda(), experts)
    offsets, rows, place = ref.expert_sort(ids, experts)
    assert order.offsets.tolist() == offsets
    assert order.order.tolist() == rows
    assert order.place.shape == ids.shape and order.place.flatten().tolist() == place
    assert order.offsets.dtype == torch.int64 and order.order.dtype == order.place.dtype == torch.int32
    return order, offsets, rows, place


@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens,choices,experts,dropped", [
    (1, 1, 1, 0), (1, 1, 1024, 0), (3, 8, 5, 0.5), (16, 2, 64, 0), (64, 8, 128, 0.1), (33, 1, 1023, 0.2), (500, 3, 2, 0),
    (1000, 4, 1024, 0.1), (3001, 3, 37, 0.1), (5000, 8, 256, 0), (7, 5, 3, 1.0), (0, 2, 4, 0), (4, 0, 4, 0)])
def test_sort(tokens, choices, experts, dropped, kind):
    _sorted(_ids(tokens, choices, experts, dropped, kind), experts)


@pytest.mark.parametrize("skew", [False, True])
@pytest.mark.parametrize("tokens,choices,experts", [(32768, 8, 512), (100003, 1, 60), (16384, 2, 1024)])
def test_sort_of_many(tokens, choices, experts, skew):
    """Runs of many entries a warp; against torch's stable sort."""
    ids = _ids(tokens, choices, experts, 0.05, skew=skew).cuda()
    order = sc.expert_sort(ids, experts)
    key = torch.where((ids >= 0) & (ids < experts), ids, experts).flatten()
    want = torch.argsort(key, stable=True)
    assert torch.equal(order.order.long(), want)
    assert torch.equal(order.place.flatten()[want].long(), torch.arange(len(want), device="cuda"))
    assert torch.equal(order.offsets, torch.searchsorted(key[want], torch.arange(experts + 1, device="cuda")))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dropped", [0, 0.3])
@pytest.mark.parametrize("tokens,choices,experts,dim", [
    (1, 1, 1, 1), (5, 3, 4, 8), (40, 2, 8, 33), (17, 5, 9, 64), (33, 8, 16, 200), (20, 9, 16, 1000), (9, 2, 4, 2047),
    (6, 4, 4, 4096), (3, 1, 7, 9001)])
def test_rows_there_and_back(tokens, choices, experts, dim, dropped, dtype):
    ids = _ids(tokens, choices, experts, dropped)
    order, offsets, rows, place = _sorted(ids, experts)
    x, y = _normal(tokens, dim, dtype=dtype), _normal(tokens * choices, dim, seed=1, dtype=dtype)
    y[offsets[-1]:] = float("nan")  # rows of no expert are not read
    dout, w = _normal(tokens, dim, seed=2, dtype=dtype), torch.rand(tokens, choices)
    got = sc.expert_gather(x.cuda(), order)
    assert torch.equal(got.cpu(), ref.expert_rows(x, rows, offsets, choices))
    r = ref.expert_combine(y, place, offsets[-1], tokens, choices)
    ref.check("dx", sc.expert_gather_grad(y.cuda(), order), r["out"])
    ref.check("sum", sc.expert_combine(y.cuda(), order), r["out"])
    for weights in (w, w.to(dtype)):
        r = ref.expert_combine(y, place, offsets[-1], tokens, choices, weights, dout)
        ref.check("out", sc.expert_combine(y.cuda(), order, weights.cuda()), r["out"])
        g = sc.expert_combine_grad(dout.cuda(), y.cuda(), order, weights.cuda())
        assert g["weights"].dtype == weights.dtype
        ref.check("dy", g["y"], r["dy"])
        ref.check("dweights", g["weights"], r["dweights"])
        assert (g["y"][offsets[-1]:] == 0).all()
        again = sc.expert_combine_grad(dout.cuda(), y.cuda(), order, weights.cuda())
        assert torch.equal(g["weights"], again["weights"])
    g = sc.expert_combine_grad(dout.cuda(), y.cuda(), order)
    assert set(g) == {"y"}
    ref.check("dy, no weights", g["y"], ref.expert_combine(y, place, offsets[-1], tokens, choices, None, dout)["dy"])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,choices,experts,dim", [
    (9001, 2, 40, 64), (12001, 1, 5, 8), (3001, 8, 16, 200), (2501, 3, 9, 1000), (1501, 32, 40, 72), (1301, 2, 4, 4096)])
def test_more_tokens_than_the_machine_holds(tokens, choices, experts, dim, dtype):
    """Several tokens for every team of threads, their rows through the ring; the same bits again."""
    ids = _ids(tokens, choices, experts, 0.1)
    order = sc.expert_sort(ids.cuda(), experts)
    place, kept = order.place.flatten().tolist(), int(order.offsets[-1])
    y, dout = _normal(tokens * choices, dim, dtype=dtype), _normal(tokens, dim, seed=2, dtype=dtype)
    y[kept:] = float("nan")
    w = torch.rand(tokens, choices)
    r = ref.expert_combine(y, place, kept, tokens, choices, w, dout)
    plain = ref.expert_combine(y, place, kept, tokens, choices, None, dout)
    y, dout, w = y.cuda(), dout.cuda(), w.cuda()
    out, dx = sc.expert_combine(y, order, w), sc.expert_gather_grad(y, order)
    ref.check("out", out, r["out"])
    ref.check("dx", dx, plain["out"])
    g, g1 = sc.expert_combine_grad(dout, y, order, w), sc.expert_combine_grad(dout, y, order)
    ref.check("dy", g["y"], r["dy"])
    ref.check("dweights", g["weights"], r["dweights"])
    ref.check("dy, no weights", g1["y"], plain["dy"])
    again = sc.expert_combine_grad(dout, y, order, w)
    assert torch.equal(sc.expert_combine(y, order, w), out) and all(torch.equal(g[k], again[k]) for k in g)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset,dim", [(0, 64), (1, 64), (8, 72), (3, 37)])
def test_slices(offset, dim, dtype):
    """Columns of wider rows, aligned or not; what lies beside them stays."""
    ids = _ids(50, 2, 6, 0.1)
    order, offsets, rows, place = _sorted(ids, 6)
    wide, wide_rows = _normal(50, 90, dtype=dtype).cuda(), _normal(100, 90, seed=1, dtype=dtype).cuda()
    at = slice(offset, offset + dim)
    x, y, w = wide[:, at], wide_rows[:, at], torch.rand(50, 2).cuda()

    def into(n, call):
        out = torch.full((n, 90), -7.0, dtype=dtype, device="cuda")
        call(out[:, at])
        assert (out[:, :offset] == -7).all() and (out[:, offset + dim:] == -7).all()
        return out[:, at]

    same = [(into(100, lambda o: sc.expert_gather(x, order, out=o)), sc.expert_gather(x.contiguous(), order)),
            (into(50, lambda o: sc.expert_gather_grad(y, order, out=o)), sc.expert_gather_grad(y.contiguous(), order)),
            (into(50, lambda o: sc.expert_combine(y, order, w, out=o)), sc.expert_combine(y.contiguous(), order, w))]
    assert all(torch.equal(a, b) for a, b in same)
    a, b = sc.expert_combine_grad(x, y, order, w), sc.expert_combine_grad(x.contiguous(), y.contiguous(), order, w)
    assert torch.equal(a["y"], b["y"])
    r = ref.expert_combine(y.cpu(), place, offsets[-1], 50, 2, w.cpu(), x.cpu())
    ref.check("dweights", a["weights"], r["dweights"])


def test_more_than_2_31_elements():
    """Offsets beyond 32 bits: the last tokens and rows."""
    ids = _ids(70000, 8, 64, 0.1)[:, :8].cuda()
    order = sc.expert_sort(ids, 64)
    x = torch.randn(70000, 4096, dtype=torch.bfloat16, device="cuda")
    rows = sc.expert_gather(x, order)
    kept = int(order.offsets[-1])
    at = torch.arange(kept - 500, kept, device="cuda")
    assert torch.equal(rows[at], x[order.order[at].long() // 8]) and (rows[kept:] == 0).all()
    w = torch.rand(70000, 8, device="cuda")
    out, g = sc.expert_combine(rows, order, w), sc.expert_combine_grad(x, rows, order, w)
    live = order.place[-500:] < kept
    share = torch.where(live, w[-500:], 0.0)
    # every row of a token is the token itself
    r = x[-500:].double() * share.double().sum(1, keepdim=True)
    assert ((out[-500:].double() - r).abs() <= (2 ** -8 + 16 * ref.EPS) * r.abs() + ref.TINY[x.dtype]).all()
    entry = order.order[at].long()
    want = (x[entry // 8].float() * w.flatten()[entry][:, None]).to(x.dtype)
    assert torch.equal(g["y"][at], want)
    square = (x[-500:].double() ** 2).sum(1, keepdim=True)
    assert ((g["weights"][-500:] - torch.where(live, square, 0.0)).abs() <= 4098 * ref.EPS * square).all()


def test_places_outside_are_passed_over():
    ids = _ids(20, 2, 5, 0)
    order, offsets, rows, place = _sorted(ids, 5)
    bad = order.place.clone()
    bad[3, 1], bad[7, 0] = -1, 40
    wrong = order._replace(place=bad)
    x, y = _normal(20, 24).cuda(), _normal(40, 24, seed=1).cuda()
    out = torch.full((40, 24), -7.0, device="cuda")
    sc.expert_gather(x, wrong, out=out)
    skipped = [place[7], place[14]]
    assert (out[skipped] == -7).all()
    keep = [i for i in range(40) if i not in skipped]
    assert torch.equal(out[keep], sc.expert_gather(x, order)[keep])
    z = y.clone()
    z[skipped] = 0
    assert torch.equal(sc.expert_combine(y, wrong), sc.expert_combine(z, order))


def test_a_token_may_choose_an_expert_twice():
    ids = torch.tensor([[2, 2], [0, 2]])
    order, *_ = _sorted(ids, 3)
    x = _normal(2, 16).cuda()
    assert torch.equal(sc.expert_gather_grad(sc.expert_gather(x, order), order), 2 * x)


def test_nothing_to_do():
    for shape in ((0, 2), (3, 0)):
        order, *_ = _sorted(torch.zeros(shape, dtype=torch.int64), 4)
        x, y = torch.ones(shape[0], 8, device="cuda"), torch.ones(0, 8, device="cuda")
        assert sc.expert_gather(x, order).shape == (0, 8)
        out = sc.expert_combine(y, order, torch.ones(shape, device="cuda"))
        assert out.shape == (shape[0], 8) and (out == 0).all()
        assert sc.expert_combine_grad(x, y, order, torch.ones(shape, device="cuda"))["weights"].shape == shape
    order, *_ = _sorted(torch.zeros(3, 2, dtype=torch.int64), 4)
    g = sc.expert_combine_grad(torch.ones(3, 0, device="cuda"), torch.ones(6, 0, device="cuda"), order, torch.ones(3, 2, device="cuda"))
    assert (g["weights"] == 0).all()


def test_refusals():
    ids = torch.zeros(4, 2, dtype=torch.int64, device="cuda")
    for bad, n in ((ids.float(), 4), (ids[:, :1], 4), (ids.flatten(), 4), (ids.cpu(), 4), (ids, 0), (ids, 1025)):
        with pytest.raises(ValueError):
            sc.expert_sort(bad, n)
    order = sc.expert_sort(ids, 4)
    x, y, w = torch.zeros(4, 8, device="cuda"), torch.zeros(8, 8, device="cuda"), torch.zeros(4, 2, device="cuda")
    calls = [lambda: sc.expert_gather(x[:3], order), lambda: sc.expert_gather(x.double(), order),
             lambda: sc.expert_gather(x, order, out=y[:7]), lambda: sc.expert_gather_grad(y[:7], order),
             lambda: sc.expert_combine(y, order, w[:3]), lambda: sc.expert_combine(y, order, w.half()),
             lambda: sc.expert_combine(y.cpu(), order), lambda: sc.expert_combine_grad(x[:3], y, order, w),
             lambda: sc.expert_combine_grad(x.half(), y, order, w),
             lambda: sc.expert_gather(x, order._replace(place=order.place.long())),
             lambda: sc.expert_gather(x, order._replace(offsets=order.offsets.int()))]
    for call in calls:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(sc.ScanError):
        sc.expert_gather(y[:4], order, out=y)


def test_streams_and_graphs():
    """On another stream; the whole way captured, replayed with other experts."""
    ids = _ids(300, 4, 32, 0.1).cuda()
    x, y, w = _normal(300, 256).cuda(), _normal(1200, 256, seed=1).cuda(), torch.rand(300, 4).cuda()

    def all_of():
        order = sc.expert_sort(ids, 32)
        g = sc.expert_combine_grad(x, y, order, w)
        return [*order, sc.expert_gather(x, order), sc.expert_gather_grad(y, order), sc.expert_combine(y, order, w), *g.values()]

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
    ids.copy_(ids.flip(0))
    want = all_of()
    for _ in range(2):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(made, want))
