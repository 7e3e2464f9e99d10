"""Token embedding and its gradient against float64."""
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


def _ids(kind, tokens, vocab, gen, dtype=torch.int64):
    if kind == "uniform":
        ids = torch.randint(0, vocab, (tokens,), generator=gen)
    elif kind == "one":
        ids = torch.full((tokens,), vocab - 1)
    elif kind == "few":      # runs of every length around the pieces' 128
        ids = torch.repeat_interleave(torch.arange(tokens), torch.randint(1, 300, (tokens,), generator=gen))[:tokens] % vocab
        ids = ids[torch.randperm(tokens, generator=gen)]
    else:                    # outside: a third of the entries outside [0, vocab), the types' extremes among them
        ids = torch.randint(0, vocab, (tokens,), generator=gen)
        far = torch.tensor([-1, vocab, vocab + 7, torch.iinfo(dtype).min, torch.iinfo(dtype).max])
        pick = torch.rand(tokens, generator=gen) < 1 / 3
        ids = torch.where(pick, far[torch.randint(0, 5, (tokens,), generator=gen)], ids)
    return ids.to(dtype)


def _check_grad(got, ids, dout, vocab, scale, base=None):
    total, size, counts = ref.embed_grad(ids, dout, vocab, scale)
    if base is not None:
        total, size = total + base.double(), size + base.double().abs()
    # (count + 2) roundings of partial sums and products
    ref.check("dweight", got, total, size * (counts[:, None] + 2), got.dtype, -4, 1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [1, 7, 64, 1000, 2056, 4100])
@pytest.mark.parametrize("tokens", [1, 5, 300])
def test_lookup(tokens, dim, dtype):
    gen = torch.Generator().manual_seed(tokens + dim)
    weight = torch.randn(50, dim, generator=gen).to(dtype)
    for ids_type in (torch.int32, torch.int64):
        ids = _ids("outside", tokens, 50, gen, ids_type)
        got = sc.embed(ids.cuda(), weight.cuda(), 3.5)
        want = ref.embed(ids, weight, 3.5)
        assert torch.equal(got.cpu(), (want.float()).to(dtype))  # one float32 product, rounded once


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [1, 72, 100, 2056])
@pytest.mark.parametrize("kind", ["uniform", "one", "few", "outside"])
@pytest.mark.parametrize("tokens,vocab", [(1, 1), (3, 1000), (128, 3), (129, 70000), (2048, 33), (5003, 501)])
def test_gradient(tokens, vocab, kind, dim, dtype):
    gen = torch.Generator().manual_seed(tokens * 31 + vocab + dim)
    ids = _ids(kind, tokens, vocab, gen)
    dout = torch.randn(tokens, dim, generator=gen).to(dtype)
    if vocab * dim > 1 << 24:
        pytest.skip("the float64 reference would be large")
    got = sc.embed_grad(ids.cuda(), dout.cuda(), vocab, 0.5)
    assert got.dtype == dtype
    _check_grad(got, ids, dout, vocab, 0.5)
    wide = sc.embed_grad(ids.int().cuda() if kind != "outside" else ids.cuda(), dout.cuda(), vocab, 0.5,
                         out=torch.full((vocab, dim), 7.0, device="cuda"))
    _check_grad(wide, ids, dout, vocab, 0.5)


@pytest.mark.parametrize("tokens", [40000, 300001])
def test_gradient_of_many_tokens(tokens):
    """More sort tiles than a placement folds by itself; two, and three, digit passes."""
    gen = torch.Generator().manual_seed(tokens)
    for vocab in (1000, 70000, (1 << 20) + 5):
        ids = torch.where(torch.rand(tokens, generator=gen) < 0.3, torch.tensor(vocab - 1),
                          torch.randint(0, vocab, (tokens,), generator=gen))
        dout = torch.randn(tokens, 8, generator=gen).to(torch.bfloat16)
        _check_grad(sc.embed_grad(ids.cuda(), dout.cuda(), vocab), ids, dout, vocab, 1.0)


def test_gradient_is_the_same_on_every_run():
    gen = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(0, 50, (20000,), generator=gen, device="cuda")
    dout = torch.randn(20000, 130, generator=gen, device="cuda")
    first = sc.embed_grad(ids, dout, 50)
    assert all(torch.equal(first, sc.embed_grad(ids, dout, 50)) for _ in range(5))


def test_accumulate_strides_and_shapes():
    gen = torch.Generator().manual_seed(2)
    ids = _ids("outside", 600, 40, gen).reshape(3, 200)
    dout = torch.randn(3, 200, 24, generator=gen).to(torch.bfloat16)
    base = torch.randn(40, 24, generator=gen)
    out = base.cuda()
    assert sc.embed_grad(ids.cuda(), dout.cuda(), 40, 2.0, out=out, accumulate=True) is out
    _check_grad(out, ids, dout, 40, 2.0, base)
    absent = torch.ones(40, dtype=torch.bool)
    absent[ids.flatten()[(ids.flatten() >= 0) & (ids.flatten() < 40)]] = False
    assert torch.equal(out.cpu()[absent], base[absent])
    # rows inside a wider, unaligned buffer, on both sides
    wide_w, wide_o = torch.randn(40, 37, generator=gen).cuda(), torch.full((40, 31), -7.0, device="cuda")
    got = sc.embed(ids.cuda(), wide_w[:, 5:29])
    assert got.shape == (3, 200, 24)
    assert torch.equal(got.cpu(), ref.embed(ids, wide_w[:, 5:29].cpu(), 1.0).float())
    wide_d = torch.randn(600, 31, generator=gen)
    sc.embed_grad(ids.flatten().cuda(), wide_d.cuda()[:, 3:27], 40, out=wide_o[:, 1:25])
    _check_grad(wide_o[:, 1:25], ids, wide_d[:, 3:27], 40, 1.0)
    assert (wide_o[:, 0] == -7).all() and (wide_o[:, 25:] == -7).all()


def test_empty_and_nothing_inside():
    w = torch.randn(10, 16, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert sc.embed(none, w).shape == (0, 16)
    assert (sc.embed_grad(none, torch.empty(0, 16, device="cuda"), 10, out=torch.ones(10, 16, device="cuda")) == 0).all()
    outside = torch.full((300,), -1, device="cuda")
    assert (sc.embed_grad(outside, torch.randn(300, 16, device="cuda"), 10) == 0).all()
    assert (sc.embed(outside, w) == 0).all()


def test_infinities_stay_in_their_rows():
    """A masked token's row may hold anything; so may the weight rows nobody looks up."""
    ids = torch.tensor([3, -1, 3, 5], device="cuda")
    dout = torch.ones(4, 16, device="cuda")
    dout[1] = float("nan")
    got = sc.embed_grad(ids, dout, 8)
    assert torch.isfinite(got).all() and (got[3] == 2).all() and (got[5] == 1).all()
    w = torch.full((8, 16), float("nan"), device="cuda")
    w[[3, 5]] = 1.0
    assert (sc.embed(ids, w)[[0, 2, 3]] == 1).all() and (sc.embed(ids, w)[1] == 0).all()


def test_offsets_past_32_bits():
    vocab, dim = 70000, 32768  # 2.3e9 elements
    w = torch.zeros(vocab, dim, dtype=torch.bfloat16, device="cuda")
    w[vocab - 1] = 3.0
    ids = torch.tensor([vocab - 1, 0, vocab - 1], device="cuda")
    assert (sc.embed(ids, w)[[0, 2]] == 3).all()
    sc.embed_grad(ids, torch.ones(3, dim, dtype=torch.bfloat16, device="cuda"), vocab, out=w)
    assert (w[vocab - 1] == 2).all() and (w[0] == 1).all() and (w[1:vocab - 1] == 0).all()


def test_on_another_stream():
    s = torch.cuda.Stream()
    ids = torch.arange(1000, device="cuda") % 7
    dout = torch.ones(1000, 64, device="cuda")
    torch.cuda.synchronize()
    got = sc.embed_grad(ids, dout, 7, stream=s)
    x = torch.arange(100000, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    y = sc.scan_exclusive(x, stream=s)  # the look-back area after the scratch of another call
    s.synchronize()
    assert torch.equal(got[:, 0].cpu(), torch.bincount(ids.cpu(), minlength=7).float())
    assert torch.equal(y.cpu(), (x.cpu().cumsum(0) - x.cpu()).int())
    assert sc.sc_get_device_error(s.cuda_stream) == sc.SC_OK


def test_refusals():
    ids = torch.zeros(3, dtype=torch.int64, device="cuda")
    w = torch.zeros(5, 8, device="cuda")
    for bad in (lambda: sc.embed(ids.cpu(), w), lambda: sc.embed(ids.float(), w), lambda: sc.embed(ids, w.double()),
                lambda: sc.embed(ids, w.cpu()), lambda: sc.embed(ids, w.t()), lambda: sc.embed(ids, w[0]),
                lambda: sc.embed(ids, w, out=torch.zeros(3, 7, device="cuda")),
                lambda: sc.embed_grad(ids, w, 5), lambda: sc.embed_grad(ids, w[:3], -1),
                lambda: sc.embed_grad(ids, w[:3], 5, accumulate=True),
                lambda: sc.embed_grad(ids, w[:3], 5, out=torch.zeros(5, 8, device="cuda", dtype=torch.float16))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(sc.ScanError):
        sc.embed_grad(ids, w[:3], 5, out=w)  # dweight over dout
