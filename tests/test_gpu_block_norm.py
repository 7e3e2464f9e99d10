"""The norm of a token's channels and its gradient against float64."""
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


def _cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _run(x, weight, bias, rms, residual, dy, dsum, eps=1e-5, flat=True):
    """Outputs and gradients as rows x channels."""
    dev = _cuda(x, weight, bias, residual, dy, dsum)
    return _run_dev(*dev[:3], rms, *dev[3:], eps=eps)


def _run_dev(x, weight, bias, rms, residual, dy, dsum, eps=1e-5):
    saved = sc.layer_norm_saved(x)
    y = sc.layer_norm(x, weight, bias, eps, rms, residual, saved=saved)
    s = x
    if residual is not None:
        y, s = y
    g = sc.layer_norm_grad(dy, s, weight, bias, rms, saved=saved, dsum=dsum)
    assert set(g) == {"x"} | ({"weight"} if weight is not None else set()) | ({"bias"} if bias is not None else set())
    return y, s, saved, g


def _check(x, weight, bias, rms, residual, dy, dsum, got, eps=1e-5):
    ch = x.shape[-1]
    flat = [None if t is None else t.reshape(-1, ch) for t in (x, residual, dy, dsum)]
    r = ref.norm(flat[0], weight, bias, eps, rms, flat[1], flat[2], flat[3])
    y, s, saved, g = got
    assert torch.equal(s.cpu().reshape(-1, ch).double(), r["sum"][0])
    assert s.dtype == y.dtype == g["x"].dtype == x.dtype
    ref.check("mean", saved.reshape(-1, 2)[:, :1], r["mean"])
    ref.check("r", saved.reshape(-1, 2)[:, 1:], r["r"])
    ref.check("y", y.reshape(-1, ch), r["y"])
    ref.check("dx", g["x"].reshape(-1, ch), r["dx"])
    for k in ("weight", "bias"):
        if k in g:
            assert g[k].dtype == torch.float32
            ref.check("d" + k, g[k], r["d" + k])


# a lane's part of a warp, a warp, CTAs of 256 to 1024 threads, and rows read again;
# by vectors and, odd ones, by elements
WIDTHS = [1, 3, 8, 32, 63, 64, 100, 128, 136, 256, 257, 512, 520, 1000, 1024, 2047, 2048, 4096, 4104, 5001, 8192, 8193,
          8200, 16384, 20001]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("channels", WIDTHS)
def test_forward_and_gradient(channels, rms, dtype):
    rows = 1 if channels > 8192 else 5 if channels > 600 else 37
    x, dy = _normal(rows, channels, dtype=dtype), _normal(rows, channels, seed=1, dtype=dtype)
    w, b = 1 + _normal(channels, seed=2, dtype=dtype, scale=0.1), _normal(channels, seed=3, dtype=dtype)
    res, ds = _normal(rows, channels, seed=4, dtype=dtype, scale=3.0), _normal(rows, channels, seed=5, dtype=dtype)
    _check(x, w, b, rms, res, dy, ds, _run(x, w, b, rms, res, dy, ds))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("weight,bias,wide,residual,dsum", [
    (False, False, False, False, False), (True, False, False, False, True), (False, True, True, True, False),
    (True, True, True, False, False), (True, False, True, True, True)])
def test_what_is_left_out(weight, bias, wide, residual, dsum, dtype):
    """Without weight, bias, residual; parameters in float32 beside 16-bit rows."""
    kind = torch.float32 if wide else dtype
    for channels in (72, 1001):
        x, dy = _normal(2, 9, channels, dtype=dtype), _normal(2, 9, channels, seed=1, dtype=dtype)
        w = _normal(channels, seed=2, dtype=kind) if weight else None
        b = _normal(channels, seed=3, dtype=kind) if bias else None
        res = _normal(2, 9, channels, seed=4, dtype=dtype) if residual else None
        ds = _normal(2, 9, channels, seed=5, dtype=dtype) if dsum else None
        _check(x, w, b, False, res, dy, ds, _run(x, w, b, False, res, dy, ds))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,channels", [(20011, 64), (7001, 33), (3001, 520), (1501, 2056), (700, 4097)])
def test_more_rows_than_the_machine_holds(rows, channels, dtype):
    """Several rows for every CTA of the gradient; the same bits again."""
    x, dy = _normal(rows, channels, dtype=dtype), _normal(rows, channels, seed=1, dtype=dtype)
    w, b = _normal(channels, seed=2, dtype=dtype), _normal(channels, seed=3, dtype=dtype)
    got = _run(x, w, b, False, None, dy, None)
    _check(x, w, b, False, None, dy, None, got)
    again = _run(x, w, b, False, None, dy, None)
    assert torch.equal(got[0], again[0]) and all(torch.equal(got[3][k], again[3][k]) for k in got[3])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset,channels", [(0, 64), (1, 64), (64, 64), (3, 37)])
def test_slices_and_strides(offset, channels, dtype):
    """Columns of wider rows, aligned or not, rows in another order, a row used for all."""
    joint = _normal(3, 20, 130, dtype=dtype)
    x = joint[:, :, offset:offset + channels]
    dev = joint.cuda()[:, :, offset:offset + channels]
    w, dy = _normal(channels, seed=2, dtype=dtype), _normal(3, 20, channels, seed=1, dtype=dtype)
    _check(x, w, None, False, None, dy, None, _run_dev(dev, *_cuda(w), None, False, None, *_cuda(dy), None))
    out = torch.full((3, 20, 130), -7.0, dtype=dtype, device="cuda")
    y = sc.layer_norm(dev, w.cuda(), out=out[:, :, offset:offset + channels])
    assert (out[:, :, :offset] == -7).all() and (out[:, :, offset + channels:] == -7).all()
    # aligned rows and others are summed in different orders: the definition's bound, not the same bits
    want = [v.view(3, 20, channels) for v in ref.norm(x.reshape(-1, channels), w)["y"]]
    ref.check("columns", y, want)
    ref.check("rows turned", sc.layer_norm(dev.transpose(0, 1), w.cuda()), [v.transpose(0, 1) for v in want])
    ref.check("one row", sc.layer_norm(dev[:1, :1].expand(4, 5, channels), w.cuda()), [v[:1, :1].expand(4, 5, channels) for v in want])
    four = dev.reshape(3, 4, 5, channels)
    got = sc.layer_norm(four, residual=four)
    flat = sc.layer_norm(dev, residual=dev)
    assert all(torch.equal(a.reshape(3, 20, channels), b) for a, b in zip(got, flat))


def test_more_than_2_31_elements():
    """Offsets beyond 32 bits: the last rows as a call of their own has them, bit by bit."""
    x = torch.randn(540000, 4096, dtype=torch.bfloat16, device="cuda")
    w = torch.randn(4096, device="cuda")
    saved, few = sc.layer_norm_saved(x), sc.layer_norm_saved(x[-1000:])
    y, s = sc.layer_norm(x, w, residual=x, saved=saved)
    y2, s2 = sc.layer_norm(x[-1000:], w, residual=x[-1000:], saved=few)
    assert torch.equal(y[-1000:], y2) and torch.equal(s[-1000:], s2) and torch.equal(saved[-1000:], few)
    del y
    dx = sc.layer_norm_grad(x, s, w, saved=saved, dsum=x)["x"]
    assert torch.equal(dx[-1000:], sc.layer_norm_grad(x[-1000:], s2, w, saved=few, dsum=x[-1000:])["x"])


def test_strides_that_two_cannot_tell():
    x = torch.zeros(4, 5, 6, 8, device="cuda").transpose(0, 1).transpose(1, 2)
    with pytest.raises(ValueError, match="strides"):
        sc.layer_norm(x[::2, ::2, ::2])


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_residual_is_a_sum_and_then_a_norm(dtype):
    x, res = _cuda(_normal(40, 256, dtype=dtype), _normal(40, 256, seed=1, dtype=dtype, scale=8.0))
    y, s = sc.layer_norm(x, residual=res)
    assert torch.equal(s, x + res) and torch.equal(y, sc.layer_norm(x + res))


@pytest.mark.parametrize("channels", [16, 300, 4096, 9000])
def test_rows_far_from_zero_and_rows_of_one_value(channels):
    """The variance is of the centred row: a mean of 1000 deviations costs the digits of
    the mean, not of its square; a constant row gives the bias."""
    x = _normal(4, channels, scale=0.1) + 100.0
    b = _normal(channels, seed=1)
    dy = _normal(4, channels, seed=2)
    _check(x, None, b, False, None, dy, None, _run(x, None, b, False, None, dy, None))
    same = torch.full((3, channels), 0.75, device="cuda")  # its sums are exact in any order
    assert torch.equal(sc.layer_norm(same, None, b.cuda()), b.cuda().expand(3, channels))
    zero = torch.zeros(3, channels, device="cuda")
    assert (sc.layer_norm(zero, rms=True) == 0).all()


def test_an_infinity_or_nan_stays_in_its_row():
    for channels in (24, 512, 3000, 9000):
        x = _normal(6, channels)
        clean = sc.layer_norm(x.cuda())
        x[1, 3], x[4, channels - 1] = float("inf"), float("nan")
        y = sc.layer_norm(x.cuda())
        rows = [0, 2, 3, 5]
        assert torch.equal(y[rows], clean[rows]) and y[1].isnan().any() and y[4].isnan().all()


def test_nothing_to_do():
    x = torch.zeros(0, 5, 8, device="cuda")
    w = torch.ones(8, device="cuda")
    saved = sc.layer_norm_saved(x)
    assert sc.layer_norm(x, w, saved=saved).shape == x.shape
    g = sc.layer_norm_grad(x, x, w, w, saved=saved)
    assert g["x"].shape == x.shape and (g["weight"] == 0).all() and (g["bias"] == 0).all()
    none = torch.zeros(3, 0, device="cuda")
    assert sc.layer_norm(none).shape == (3, 0)
    assert sc.layer_norm(torch.ones(8, device="cuda")).shape == (8,)


def test_refusals():
    x, w = torch.zeros(4, 8, device="cuda"), torch.zeros(8, device="cuda")
    saved = sc.layer_norm_saved(x)
    for bad in (dict(weight=w[:7]), dict(weight=w.half()), dict(weight=w, bias=w.bfloat16()), dict(eps=-1.0),
                dict(eps=float("nan")), dict(residual=x[:3]), dict(residual=x.half()), dict(out=x.half()),
                dict(saved=saved[:2]), dict(weight=w.cpu())):
        with pytest.raises(ValueError):
            sc.layer_norm(x, **bad)
    with pytest.raises(ValueError):
        sc.layer_norm(x.double())
    with pytest.raises(ValueError):
        sc.layer_norm(x.cpu())
    with pytest.raises(sc.ScanError):
        sc.layer_norm(x, out=x)
    with pytest.raises(ValueError, match="saved"):
        sc.layer_norm_grad(x, x, w)


def test_streams_and_graphs():
    """On another stream than the inputs'; captured and replayed with other inputs.  The
    gradient's sums over tokens need scratch memory: refused while a stream captures."""
    x, w = _cuda(_normal(300, 1024, dtype=torch.bfloat16), _normal(1024, dtype=torch.bfloat16))
    want = sc.layer_norm(x, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sc.layer_norm(x, w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    dy, saved = torch.ones_like(x), sc.layer_norm_saved(x)
    sc.layer_norm(x, w, saved=saved)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = sc.layer_norm(x, w, saved=saved)
        dx = sc.layer_norm_grad(dy, x, saved=saved)["x"]
        with pytest.raises(sc.ScanError):
            sc.layer_norm_grad(dy, x, w, saved=saved)
    x.copy_(x.flip(0))
    g.replay()
    assert torch.equal(y, want.flip(0)) and torch.equal(dx, sc.layer_norm_grad(dy, x, saved=saved)["x"])
