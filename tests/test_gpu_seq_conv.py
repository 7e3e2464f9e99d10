"""Causal convolution, its gradient and its single-token form against float64."""
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


def _case(batch, length, channels, width, dtype, packed, seed=0):
    gen = torch.Generator().manual_seed(seed + batch * 1000 + length * 10 + channels + width)

    def normal(*shape):
        return torch.randn(*shape, generator=gen).to(dtype)

    heads = torch.rand(batch, length, generator=gen) < 0.2 if packed else None
    state = normal(batch, width - 1, channels) if packed else None
    return normal(batch, length, channels), normal(channels, width), normal(channels), heads, state, \
        normal(batch, length, channels)


def _cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _check_all(case, act, got_y, got_final, grads):
    x, w, b, heads, state, dy = case
    r = ref.conv(x, w, b, heads, state, act, dy)
    width, dtype, tokens = w.shape[1], x.dtype, x.shape[0] * x.shape[1]
    # pre is a sum of width + 1 terms; length 0 in the bound: no recurrence
    ref.check("y", got_y, r["y"], r["size"] + r["y"].abs(), dtype, 0, width + 1)
    assert torch.equal(got_final.cpu(), r["final"].to(dtype))
    if grads is None:
        return
    ref.check("dx", grads["x"], r["dx"], r["dx_size"], dtype, 0, width + 1)
    ref.check("dweight", grads["weight"], r["dweight"], r["dweight_size"], torch.float32, 0, tokens)
    ref.check("dbias", grads["bias"], r["dbias"], r["dbias_size"], torch.float32, 0, tokens)
    if state is not None:
        ref.check("dstate", grads["state"], r["dstate"], r["dstate_size"], dtype, 0, width + 1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("width", [1, 2, 3, 4, 5, 8])
@pytest.mark.parametrize("batch,length,channels", [(1, 1, 1), (2, 2, 64), (3, 3, 33), (1, 130, 1000), (2, 41, 520)])
def test_forward_and_gradient(batch, length, channels, width, packed, dtype):
    case = _case(batch, length, channels, width, dtype, packed)
    x, w, b, heads, state, dy = _cuda(*case)
    final = torch.empty(batch, width - 1, channels, dtype=dtype, device="cuda")
    y = sc.causal_conv(x, w, b, heads=heads, state=state, final_state=final)
    _check_all(case, True, y, final, sc.causal_conv_grad(dy, x, w, b, heads=heads, state=state))


@pytest.mark.parametrize("length", [700, 5000])
def test_long_rows_and_no_activation(length):
    case = _case(2, length, 16, 4, torch.float32, True)
    x, w, b, heads, state, dy = _cuda(*case)
    final = torch.empty(2, 3, 16, device="cuda")
    y = sc.causal_conv(x, w, b, activation=None, heads=heads, state=state, final_state=final)
    grads = sc.causal_conv_grad(dy, x, w, b, activation=None, heads=heads, state=state)
    _check_all(case, False, y, final, grads)
    again = sc.causal_conv_grad(dy, x, w, b, activation=None, heads=heads, state=state)
    assert all(torch.equal(grads[k], again[k]) for k in grads)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset,channels", [(0, 64), (1, 64), (64, 64), (3, 37)])
def test_slices_of_a_joint_buffer(offset, channels, dtype):
    """x, dy and y as columns of wider rows, aligned or not; no bias."""
    gen = torch.Generator().manual_seed(offset)
    joint = torch.randn(2, 20, 130, generator=gen).to(dtype)
    x, w, dy = joint[:, :, offset:offset + channels], torch.randn(channels, 4, generator=gen).to(dtype), \
        torch.randn(2, 20, 130, generator=gen).to(dtype)[:, :, offset:offset + channels]
    dev = joint.cuda()
    out = torch.full((2, 20, 130), -7.0, dtype=dtype, device="cuda")
    xd = dev[:, :, offset:offset + channels]
    y = sc.causal_conv(xd, w.cuda(), out=out[:, :, offset:offset + channels])
    r = ref.conv(x, w, None, dy=dy)
    ref.check("y", y, r["y"], r["size"] + r["y"].abs(), dtype, 0, 5)
    assert (out[:, :, :offset] == -7).all() and (out[:, :, offset + channels:] == -7).all()
    wide = torch.zeros(2, 20, 130, dtype=dtype, device="cuda")
    wide[:, :, offset:offset + channels] = dy.cuda()
    g = sc.causal_conv_grad(wide[:, :, offset:offset + channels], xd, w.cuda())
    ref.check("dx", g["x"], r["dx"], r["dx_size"], dtype, 0, 5)
    # y in the other columns of x's own buffer
    if offset == 0:
        y2 = sc.causal_conv(xd, w.cuda(), out=dev[:, :, 64:128])
        assert torch.equal(y2, y)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("width", [1, 2, 4, 7])
@pytest.mark.parametrize("channels", [40, 33])
def test_prompt_in_parts_and_token_by_token(channels, width, dtype):
    """A row cut anywhere gives the whole row's outputs; single tokens continue a prompt."""
    x, w, b, _, _, _ = _cuda(*_case(3, 24, channels, width, dtype, False))
    whole = sc.causal_conv(x, w, b)
    for cut in (1, 2, 23):
        mid = torch.empty(3, width - 1, channels, dtype=dtype, device="cuda")
        end = torch.empty_like(mid)
        first = sc.causal_conv(x[:, :cut], w, b, final_state=mid)
        second = sc.causal_conv(x[:, cut:], w, b, state=mid, final_state=end)
        assert torch.equal(torch.cat([first, second], 1), whole)
    pool = torch.full((5, width - 1, channels), 9.0, dtype=dtype, device="cuda")
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    mid = torch.empty(3, width - 1, channels, dtype=dtype, device="cuda")
    sc.causal_conv(x[:, :11], w, b, final_state=mid)
    pool[slots.long()] = mid
    for t in range(11, 24):
        got = sc.causal_conv_step(x[:, t], pool, w, b, slots=slots)
        # the same sums in the same order
        want = whole[:, t]
        ref.check("token", got, want, want.abs() + 10, dtype, 0, width + 1)
    assert torch.equal(pool[slots.long()], end)
    assert (pool[[1, 3]] == 9).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_step_rows_that_sit_out(dtype):
    gen = torch.Generator().manual_seed(4)
    x, w = torch.randn(6, 72, generator=gen).to(dtype), torch.randn(72, 4, generator=gen).to(dtype)
    pool = torch.randn(5, 3, 72, generator=gen).to(dtype)
    slots = torch.tensor([3, -1, 0, 5, 2**31 - 1, 1], dtype=torch.int32)
    dev = pool.cuda()
    y = sc.causal_conv_step(x.cuda(), dev, w.cuda(), slots=slots.cuda(), out=torch.full((6, 72), 5.0, dtype=dtype, device="cuda"))
    for r, slot in enumerate(slots.tolist()):
        if not 0 <= slot < 5:
            assert (y[r] == 0).all()
            continue
        one = ref.conv(x[r][None, None], w, None, state=pool[slot][None])
        ref.check("y", y[r], one["y"][0, 0], one["size"][0, 0] + one["y"][0, 0].abs(), dtype, 0, 5)
        assert torch.equal(dev[slot].cpu(), torch.cat([pool[slot][1:], x[r][None]]))
    assert torch.equal(dev[[2, 4]].cpu()[1], pool[4])


def test_infinities_of_another_segment_stay_there():
    x = torch.randn(1, 40, 64, device="cuda")
    w = torch.randn(64, 4, device="cuda")
    heads = torch.zeros(1, 40, dtype=torch.bool, device="cuda")
    heads[0, 17] = True
    want = sc.causal_conv(x, w, heads=heads)
    dy = torch.randn(1, 40, 64, device="cuda")
    g = sc.causal_conv_grad(dy, x, w, heads=heads)
    bad, dbad = x.clone(), dy.clone()
    bad[0, :17] = float("nan")
    bad[0, 16, ::2] = float("inf")
    dbad[0, 17:] = float("nan")
    assert torch.equal(sc.causal_conv(bad, w, heads=heads)[:, 17:], want[:, 17:])
    assert torch.equal(sc.causal_conv_grad(dbad, x, w, heads=heads)["x"][:, :17], g["x"][:, :17])
    short = torch.randn(64, 2, device="cuda")  # fewer taps than the kernel's registers hold
    bad = x.clone()
    bad[0, 3] = float("inf")
    assert torch.equal(sc.causal_conv(bad, short)[:, 5:], sc.causal_conv(x, short)[:, 5:])


def test_empty():
    w = torch.randn(8, 4, device="cuda")
    state = torch.randn(2, 3, 8, device="cuda")
    final = torch.empty_like(state)
    assert sc.causal_conv(torch.empty(2, 0, 8, device="cuda"), w, state=state, final_state=final).shape == (2, 0, 8)
    assert torch.equal(final, state)
    sc.causal_conv(torch.empty(2, 0, 8, device="cuda"), w, final_state=final)
    assert (final == 0).all()
    g = sc.causal_conv_grad(torch.empty(2, 0, 8, device="cuda"), torch.empty(2, 0, 8, device="cuda"), w)
    assert (g["weight"] == 0).all() and (g["bias"] == 0).all()
    assert sc.causal_conv(torch.empty(0, 5, 8, device="cuda"), w).shape == (0, 5, 8)
    assert sc.causal_conv_step(torch.empty(0, 8, device="cuda"), state, w).shape == (0, 8)


def test_offsets_past_32_bits():
    row = (1 << 31) + 64
    flat = torch.zeros(row + 64 * 8, dtype=torch.bfloat16, device="cuda")
    x = flat.as_strided((2, 8, 64), (row, 64, 1))
    x[1] = 1.0
    w = torch.ones(64, 2, dtype=torch.bfloat16, device="cuda")
    y = sc.causal_conv(x, w, activation=None)
    assert (y[0] == 0).all() and (y[1, 0] == 1).all() and (y[1, 1:] == 2).all()
    g = sc.causal_conv_grad(x, x, w, activation=None)
    assert (g["x"][1, :7] == 2).all() and (g["weight"][:, 1] == 8).all()


def test_capture_of_the_calls_without_scratch():
    x = torch.randn(2, 16, 64, device="cuda")
    w = torch.randn(64, 4, device="cuda")
    pool = torch.zeros(2, 3, 64, device="cuda")
    y, one = torch.empty_like(x), torch.empty(2, 64, device="cuda")
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        g.capture_begin()
        sc.causal_conv(x, w, out=y)
        sc.causal_conv_step(x[:, 0], pool, w, out=one)
        with pytest.raises(sc.ScanError):
            sc.causal_conv_grad(x, x, w)  # its sums need the stream's workspace
        g.capture_end()
    for turn in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, sc.causal_conv(x, w))
    assert torch.equal(pool[:, 1:], x[:, :1].expand(2, 2, 64)) and (pool[:, 0] == 0).all()


def test_refusals():
    x, w = torch.zeros(2, 4, 8, device="cuda"), torch.zeros(8, 4, device="cuda")
    for bad in (lambda: sc.causal_conv(x.cpu(), w), lambda: sc.causal_conv(x[0], w), lambda: sc.causal_conv(x, w.half()),
                lambda: sc.causal_conv(x, w[:7]), lambda: sc.causal_conv(x, torch.zeros(8, 9, device="cuda")),
                lambda: sc.causal_conv(x, w, activation="relu"), lambda: sc.causal_conv(x.transpose(1, 2), w[:4]),
                lambda: sc.causal_conv(x, w, heads=torch.zeros(2, 5, dtype=torch.bool, device="cuda")),
                lambda: sc.causal_conv(x, w, heads=torch.zeros(2, 4, device="cuda")),
                lambda: sc.causal_conv(x, w, state=torch.zeros(2, 4, 8, device="cuda")),
                lambda: sc.causal_conv(x, w, bias=torch.zeros(8, device="cuda").double()),
                lambda: sc.causal_conv_grad(x[:, :3], x, w),
                lambda: sc.causal_conv_step(x[:, 0], torch.zeros(2, 2, 8, device="cuda"), w),
                lambda: sc.causal_conv_step(x[:, 0], torch.zeros(2, 3, 8, device="cuda"), w,
                                            slots=torch.zeros(2, dtype=torch.int64, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(sc.ScanError):
        sc.causal_conv(x, w, out=x)
    with pytest.raises(sc.ScanError):  # fewer state rows than x rows, and no slots
        sc.causal_conv_step(x[:, 0], torch.zeros(1, 3, 8, device="cuda"), w)
