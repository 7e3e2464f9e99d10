"""Selective scan, its gradient and its single-token form against float64."""
import pytest
import torch

import seq_reference as ref
import stream_compaction_gb300 as sc
from gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def _case(batch, length, channels, states, groups, dtype, packed=False, gated=True, plain=False, seed=0):
    """Inputs on the CPU by name.  d lies in [0.01, 0.5], |A| in [0.1, 8]: decays from 0.999 to 0.02."""
    gen = torch.Generator().manual_seed(seed + batch + 7 * length + 13 * channels + 17 * states + groups)

    def normal(*shape, dtype=dtype, scale=1.0):
        return (torch.randn(*shape, generator=gen) * scale).to(dtype)

    c = {"x": normal(batch, length, channels), "dt": normal(batch, length, channels, scale=0.3),
         "A": -(0.1 + 7.9 * torch.rand(channels, states, generator=gen)),
         "B": normal(batch, length, groups, states), "C": normal(batch, length, groups, states)}
    if plain:
        c["dt"] = (0.01 + 0.3 * torch.rand(batch, length, channels, generator=gen)).to(dtype)
        return c, {"softplus": False}, normal(batch, length, channels)
    c["D"] = normal(channels, dtype=torch.float32)
    c["dt_bias"] = normal(channels, dtype=torch.float32, scale=0.5) - 3
    if gated:
        c["z"] = normal(batch, length, channels)
    if packed:
        c["heads"] = torch.rand(batch, length, generator=gen) < 0.1
        c["state"] = normal(batch, channels, states, dtype=torch.float32)
    return c, {}, normal(batch, length, channels)


def _dev(c):
    return {k: v.cuda() for k, v in c.items()}


def _run(c, opts, dy=None, dfinal=None):
    d = _dev(c)
    final = torch.empty(d["x"].shape[0], d["x"].shape[2], d["A"].shape[1], device="cuda")
    saved = None if dy is None else sc.selective_scan_saved(d["x"], d["A"])
    y = sc.selective_scan(**d, **opts, final_state=final, saved=saved)
    if dy is None:
        return y, final, None
    g = sc.selective_scan_grad(dy.cuda(), **d, **opts, saved=saved, dfinal_state=None if dfinal is None else dfinal.cuda())
    return y, final, g


def _check_all(c, opts, dy, got, dfinal=None):
    y, final, g = got
    kw = {**c, **opts}
    r = ref.scan(**kw, dy=dy, dfinal=dfinal)
    m = ref.scan(**kw, dy=dy, dfinal=dfinal, sizes=True)
    batch, length, channels = c["x"].shape
    states, groups, dtype = c["A"].shape[1], c["B"].shape[2], c["x"].dtype
    ref.check("y", y, r["y"], m["y"], dtype, length, states + 1)
    ref.check("final", final, r["final"], m["final"], torch.float32, length, 0)
    if g is None:
        return
    names = {"x": "dx", "dt": "ddt", "A": "dA", "B": "dB", "C": "dC", "D": "dD", "z": "dz", "dt_bias": "ddt_bias",
             "state": "dstate"}
    assert set(g) == {k for k in names if k in c}
    terms = {"A": batch * length, "D": batch * length, "dt_bias": batch * length, "B": channels // groups,
             "C": channels // groups}
    for k, v in g.items():
        ref.check("d" + k, v, r[names[k]], m[names[k]], v.dtype, length, terms.get(k, states + 1))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("batch,length,channels,states,groups", [
    (1, 1, 1, 1, 1), (2, 15, 8, 8, 1), (1, 16, 33, 16, 1), (3, 17, 64, 16, 2), (1, 50, 130, 3, 5), (2, 40, 40, 24, 1),
    (1, 33, 24, 32, 3), (2, 20, 16, 64, 1), (1, 31, 20, 33, 2), (2, 5, 160, 16, 1)])
def test_forward_and_gradient(batch, length, channels, states, groups, packed, dtype):
    c, opts, dy = _case(batch, length, channels, states, groups, dtype, packed)
    _check_all(c, opts, dy, _run(c, opts, dy))


@pytest.mark.parametrize("gated,plain", [(False, False), (True, True)])
def test_without_the_optional_parts(gated, plain):
    c, opts, dy = _case(2, 37, 40, 16, 1, torch.float32, gated=gated, plain=plain)
    dfinal = torch.randn(2, 40, 16, generator=torch.Generator().manual_seed(1))
    _check_all(c, opts, dy, _run(c, opts, dy, dfinal), dfinal)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("length,channels,states", [(200, 64, 16), (333, 20, 5), (1000, 8, 32)])
def test_split_lengths(length, channels, states, dtype):
    """Few channels: the length is cut into chunks, with segment starts in some of them."""
    assert sc.load().sc_selective_scan_workspace_bytes(1, length, channels, states, 1) > 0
    for packed in (False, True):
        c, opts, dy = _case(1, length, channels, states, 1, dtype, packed)
        if packed:  # whole chunks without a start, too
            c["heads"] &= torch.rand(1, length, generator=torch.Generator().manual_seed(3)) < 0.05
        dfinal = torch.randn(1, channels, states, generator=torch.Generator().manual_seed(2))
        got = _run(c, opts, dy, dfinal)
        _check_all(c, opts, dy, got, dfinal)
        again = _run(c, opts, dy, dfinal)
        assert torch.equal(got[0], again[0]) and all(torch.equal(got[2][k], again[2][k]) for k in got[2])


def test_wide_rows_are_not_split():
    assert sc.load().sc_selective_scan_workspace_bytes(64, 40, 512, 16, 1) == 0
    c, opts, dy = _case(64, 40, 512, 16, 1, torch.bfloat16, packed=True)
    _check_all(c, opts, dy, _run(c, opts, dy))


@pytest.mark.parametrize("where", ["first", "every", "last"])
def test_segment_starts(where):
    c, opts, dy = _case(2, 35, 40, 16, 1, torch.float32, packed=True)
    heads = torch.zeros(2, 35, dtype=torch.uint8)
    heads[:, {"first": slice(0, 1), "every": slice(None), "last": slice(34, 35)}[where]] = 200
    c["heads"] = heads
    y, final, g = _run(c, opts, dy)
    _check_all(c, opts, dy, (y, final, g))
    if where != "last":
        assert (g["state"] == 0).all()  # nothing of the initial state is left


def test_gradient_by_differences():
    """The float32 gradient along a direction against a central difference of the float64 forward."""
    c, opts, dy = _case(1, 20, 16, 16, 1, torch.float32, packed=True)
    _, _, g = _run(c, opts, dy)
    gen = torch.Generator().manual_seed(9)
    for name in g:
        v = torch.randn(c[name].shape, generator=gen).double()
        step = 1e-5
        sides = []
        for sign in (1, -1):
            moved = {**c, name: c[name].double() + sign * step * v}
            sides.append((ref.scan(**moved)["y"] * dy.double()).sum())
        slope = (sides[0] - sides[1]) / (2 * step)
        got, size = (g[name].double().cpu() * v).sum(), (g[name].double().cpu() * v).abs().sum()
        # truncation: step^2 times third derivatives of O(100) sums; float32 errors: the tests above
        assert abs(got - slope) <= 1e-4 * size + 1e-6, (name, got, slope)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset", [0, 1, 8])
def test_slices_of_joint_buffers(offset, dtype):
    c, opts, dy = _case(2, 20, 64, 16, 2, dtype, packed=True)
    d = _dev(c)
    joint = torch.zeros(2, 20, 200, dtype=dtype, device="cuda")
    xz = torch.zeros(2, 20, 200, dtype=dtype, device="cuda")
    xz[:, :, offset:offset + 64], xz[:, :, offset + 64:offset + 128] = d["x"], d["z"]
    joint[:, :, offset:offset + 32], joint[:, :, offset + 32:offset + 64] = d["B"].flatten(2), d["C"].flatten(2)
    joint[:, :, offset + 64:offset + 128] = d["dt"]
    d |= {"x": xz[:, :, offset:offset + 64], "z": xz[:, :, offset + 64:offset + 128],
          "B": joint[:, :, offset:offset + 32].unflatten(2, (2, 16)),
          "C": joint[:, :, offset + 32:offset + 64].unflatten(2, (2, 16)), "dt": joint[:, :, offset + 64:offset + 128]}
    saved = sc.selective_scan_saved(d["x"], d["A"])
    final = torch.empty(2, 64, 16, device="cuda")
    wide = torch.full((2, 20, 100), -7.0, dtype=dtype, device="cuda")
    y = sc.selective_scan(**d, saved=saved, final_state=final, out=wide[:, :, offset:offset + 64])
    _check_all(c, opts, dy, (y, final, sc.selective_scan_grad(dy.cuda(), **d, saved=saved)))
    assert (wide[:, :, :offset] == -7).all() and (wide[:, :, offset + 64:] == -7).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("states,groups", [(16, 1), (6, 2), (32, 1), (50, 2), (1, 1)])
def test_token_by_token(states, groups, dtype):
    """Single tokens continue a prompt in a pool of states, rows in any order, some sitting out."""
    c, opts, _ = _case(3, 30, 40, states, groups, dtype, packed=True)
    c.pop("heads")
    r, m = ref.scan(**c), ref.scan(**c, sizes=True)
    d = _dev(c)
    head = {k: (v[:, :13] if k in ("x", "dt", "B", "C", "z") else v) for k, v in d.items()}
    mid = torch.empty(3, 40, states, device="cuda")
    sc.selective_scan(**head, final_state=mid)
    pool = torch.full((6, 40, states), 9.0, device="cuda")
    slots = torch.tensor([5, 0, 2], dtype=torch.int32, device="cuda")
    pool[slots.long()] = mid
    rows = torch.tensor([5, -1, 0, 6, 2], dtype=torch.int32, device="cuda")   # the call's rows, two of them out
    pick = torch.tensor([0, 0, 1, 1, 2], device="cuda")
    for t in range(13, 30):
        y = sc.selective_scan_step(d["x"][pick, t], d["dt"][pick, t], d["A"], d["B"][pick, t], d["C"][pick, t], pool,
                                   D=d["D"], z=d["z"][pick, t], dt_bias=d["dt_bias"], slots=rows)
        assert (y[[1, 3]] == 0).all()
        ref.check("y", y[[0, 2, 4]], r["y"][:, t], m["y"][:, t], dtype, t, states + 1)
    ref.check("state", pool[slots.long()], r["final"], m["final"], torch.float32, 30, 0)
    assert (pool[[1, 3, 4]] == 9).all()


def test_prompt_in_parts():
    c, opts, _ = _case(2, 60, 48, 16, 1, torch.float32, packed=True)
    y, final, _ = _run(c, opts)
    r, m = ref.scan(**c), ref.scan(**c, sizes=True)
    for cut in (1, 16, 37):
        part = lambda lo, hi: {k: (v[:, lo:hi].contiguous() if k in ("x", "dt", "B", "C", "z", "heads") else v)  # noqa: E731
                               for k, v in _dev(c).items()}
        mid, end = torch.empty(2, 48, 16, device="cuda"), torch.empty(2, 48, 16, device="cuda")
        first = sc.selective_scan(**part(0, cut), final_state=mid)
        second = sc.selective_scan(**{**part(cut, 60), "state": mid}, final_state=end)
        ref.check("y", torch.cat([first, second], 1), r["y"], m["y"], torch.float32, 60, 17)
        ref.check("final", end, r["final"], m["final"], torch.float32, 60, 0)


def test_infinities_of_another_segment_stay_there():
    c, opts, dy = _case(1, 64, 64, 16, 1, torch.float32, packed=True)
    c["heads"] = torch.zeros(1, 64, dtype=torch.bool)
    c["heads"][0, 21] = True
    y, _, g = _run(c, opts, dy)
    for name in ("x", "B", "C", "z", "state"):
        bad = {k: v.clone() for k, v in c.items()}
        where = bad[name] if name == "state" else bad[name][:, :21]
        where[:] = float("nan")
        where.view(-1)[::3] = float("inf")
        got, _, _ = _run(bad, opts, dy)
        assert torch.equal(got[:, 21:], y[:, 21:]), name
    late = dy.clone()
    late[:, 21:] = float("nan")
    assert torch.equal(_run(c, opts, late)[2]["x"][:, :21], g["x"][:, :21])


def test_extreme_steps():
    """d of 0 keeps the state, a huge d clears it; no NaN from either."""
    c, opts, _ = _case(1, 20, 32, 16, 1, torch.float32, gated=False)
    c["dt"][:, 5:9] = -200.0    # softplus underflows to 0
    c["dt"][:, 12] = 1e4        # every decay is 0
    y, final, _ = _run(c, opts)
    r = ref.scan(**c)
    assert torch.isfinite(y).all()
    m = ref.scan(**c, sizes=True)
    ref.check("y", y, r["y"], m["y"], torch.float32, 20, 17)
    ref.check("final", final, r["final"], m["final"], torch.float32, 20, 0)


def test_empty():
    c, opts, _ = _case(2, 0, 16, 16, 1, torch.float32, packed=True)
    dy = torch.empty(2, 0, 16)
    y, final, g = _run(c, opts, dy, torch.ones(2, 16, 16))
    assert y.shape == (2, 0, 16) and torch.equal(final.cpu(), c["state"])
    assert (g["A"] == 0).all() and (g["D"] == 0).all() and (g["dt_bias"] == 0).all() and (g["state"] == 1).all()
    c, opts, dy = _case(0, 5, 16, 16, 1, torch.float32)
    y, _, g = _run(c, opts, dy)
    assert y.shape == (0, 5, 16) and (g["A"] == 0).all()
    none = torch.empty(0, 16, device="cuda")
    bc = torch.empty(0, 1, 16, device="cuda")
    assert sc.selective_scan_step(none, none, torch.zeros(16, 16, device="cuda"), bc, bc,
                                  torch.zeros(3, 16, 16, device="cuda")).shape == (0, 16)


def test_offsets_past_32_bits():
    row = (1 << 31) + 64
    c, opts, dy = _case(2, 20, 64, 16, 1, torch.bfloat16)
    d = _dev(c)
    flat = torch.zeros(row + 20 * 64, dtype=torch.bfloat16, device="cuda")
    x = flat.as_strided((2, 20, 64), (row, 64, 1))
    x.copy_(d["x"])
    saved = sc.selective_scan_saved(x, d["A"])
    final = torch.empty(2, 64, 16, device="cuda")
    y = sc.selective_scan(**{**d, "x": x}, saved=saved, final_state=final)
    _check_all(c, opts, dy, (y, final, sc.selective_scan_grad(dy.cuda(), **{**d, "x": x}, saved=saved)))
    # a state pool whose rows pass 2^31 elements
    pool = torch.zeros((1 << 31) // 1024 + 8, 64, 16, device="cuda")
    last = pool.shape[0] - 1
    slots = torch.tensor([last, 3], dtype=torch.int32, device="cuda")
    sc.selective_scan_step(x[:, 0], d["dt"][:, 0], d["A"], d["B"][:, 0], d["C"][:, 0], pool, slots=slots)
    assert (pool[last] != 0).any() and (pool[3] != 0).any() and (pool[last - 1] == 0).all()


def test_on_another_stream_and_after_a_scan():
    c, opts, dy = _case(1, 300, 64, 16, 1, torch.float32)
    want = _run(c, opts, dy)
    d, dyd = _dev(c), dy.cuda()
    x = torch.arange(200000, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):
        saved = sc.selective_scan_saved(d["x"], d["A"], stream=s)
        y = sc.selective_scan(**d, saved=saved, stream=s)
        cum = sc.scan_inclusive(x, stream=s)
        g = sc.selective_scan_grad(dyd, **d, saved=saved, stream=s)
        s.synchronize()
        assert torch.equal(y, want[0]) and all(torch.equal(g[k], want[2][k]) for k in g)
        assert torch.equal(cum.cpu(), x.cpu().cumsum(0).int())
    assert sc.sc_get_device_error(s.cuda_stream) == sc.SC_OK
    assert sc.sc_release_stream(s.cuda_stream) == sc.SC_OK


def test_bound_workspace():
    c, opts, _ = _case(1, 300, 64, 16, 1, torch.float32)
    need = sc.load().sc_selective_scan_workspace_bytes(1, 300, 64, 16, 1)
    want = _run(c, opts)[0]
    d = _dev(c)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    small, enough = (torch.zeros(n, dtype=torch.uint8, device="cuda") for n in (need - 1, need))
    assert sc.sc_set_workspace(small.data_ptr(), need - 1, s.cuda_stream) == sc.SC_OK
    with pytest.raises(sc.ScanError):
        sc.selective_scan(**d, stream=s)
    assert sc.sc_set_workspace(enough.data_ptr(), need, s.cuda_stream) == sc.SC_OK
    y = sc.selective_scan(**d, stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    assert sc.sc_release_stream(s.cuda_stream) == sc.SC_OK


def test_refusals():
    c, opts, dy = _case(2, 8, 16, 16, 2, torch.float32, packed=True)
    d = _dev(c)
    saved = sc.selective_scan_saved(d["x"], d["A"])
    for change in ({"x": d["x"].double()}, {"x": d["x"][0]}, {"dt": d["dt"].half()}, {"dt": d["dt"][:, :7]},
                   {"A": d["A"].half()}, {"A": d["A"][:15]}, {"B": d["B"][:, :, :, :15]}, {"C": d["C"][:, :, :1]},
                   {"B": d["B"].flatten(2)}, {"D": d["D"].half()}, {"z": d["z"][:1]}, {"dt_bias": d["dt_bias"][:3]},
                   {"heads": d["heads"].int()}, {"state": d["state"].half()}, {"x": d["x"].cpu()},
                   {"saved": saved[:, :, :, :8]}, {"out": torch.empty(2, 8, 15, device="cuda")},
                   {"x": d["x"].transpose(1, 2)}, {"final_state": d["state"].half()}):
        with pytest.raises(ValueError):
            sc.selective_scan(**{**d, **change})
    with pytest.raises(ValueError):
        sc.selective_scan_grad(dy.cuda(), **d)
    with pytest.raises(sc.ScanError):
        sc.selective_scan(**d, out=d["z"])
    with pytest.raises(sc.ScanError):
        sc.selective_scan(**d, final_state=d["state"])
    wide = {**d, "A": torch.zeros(16, 65, device="cuda"), "B": torch.zeros(2, 8, 2, 65, device="cuda"),
            "C": torch.zeros(2, 8, 2, 65, device="cuda"), "state": None}
    with pytest.raises(sc.ScanError):
        sc.selective_scan(**wide)
