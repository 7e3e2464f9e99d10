"""The block operators' part of the C ABI: structure layouts, and the argument checks
that return before any CUDA call."""
import ctypes
import os
import subprocess

import pytest

import stream_compaction_gb300 as sc
from stream_compaction_gb300 import seq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BIG = 1 << 50


@pytest.fixture(scope="module")
def lib():
    from stream_compaction_gb300 import build
    build.build()
    return sc.load()


def test_structures_match_the_header(tmp_path):
    src = tmp_path / "s.c"
    src.write_text('#include "sc_seq.h"\n#include <stdio.h>\nint main(void) { printf("%zu %zu %zu %zu %zu %zu\\n", '
                   'sizeof(sc_gated_desc), sizeof(sc_norm_desc), sizeof(sc_expert_desc), offsetof(sc_gated_desc, state), '
                   'offsetof(sc_norm_desc, bias), offsetof(sc_expert_desc, weights)); return 0; }\n')
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-I" + os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(seq.GatedDesc), ctypes.sizeof(seq.NormDesc), ctypes.sizeof(seq.ExpertDesc),
                   seq.GatedDesc.state.offset, seq.NormDesc.bias.offset, seq.ExpertDesc.weights.offset]


def gated(**k):
    base = dict(dtype=sc.SC_F32, sigmoid=1, batch=2, length=8, channels=16, x=0x10000, gate=0x20000, x_batch=128,
                x_token=16, gate_batch=128, gate_token=16, heads=0, state=0)
    return seq.GatedDesc(**{**base, **k})


def test_gated_refusals(lib):
    run = lambda d, y=0x30000, yb=128, yt=16, fs=0, saved=0: lib.sc_gated_scan(d, y, yb, yt, fs, saved, 0)  # noqa: E731
    assert lib.sc_gated_scan(None, 0x30000, 128, 16, 0, 0, 0) == sc.SC_ERR_INVALID
    for bad in (dict(batch=-1), dict(length=-1), dict(channels=-1), dict(x=0), dict(gate=0), dict(x=0x10001),
                dict(gate=0x20002), dict(x_token=-16), dict(gate_batch=-1), dict(state=0x40002), dict(dtype=-1),
                dict(dtype=12), dict(length=BIG), dict(batch=BIG)):
        assert run(gated(**bad)) == sc.SC_ERR_INVALID, bad
    assert run(gated(dtype=sc.SC_I32)) == sc.SC_ERR_UNSUPPORTED
    for bad in (dict(y=0), dict(y=0x10000), dict(y=0x20040), dict(yt=8), dict(yb=64), dict(fs=0x40002), dict(saved=0x40002),
                dict(saved=0x20000), dict(fs=0x30000), dict(saved=0x30000), dict(y=0x30002)):
        assert run(gated(), **bad) == sc.SC_ERR_INVALID, bad
    assert run(gated(state=0x40000), fs=0x40000) == sc.SC_ERR_INVALID
    assert run(gated(heads=0x50000), y=0x50000) == sc.SC_ERR_INVALID
    assert run(gated(batch=0)) == sc.SC_OK
    assert run(gated(channels=0)) == sc.SC_OK
    base = dict(dy=0x30000, db=128, dt=16, saved=0x40000, df=0, dx=0x50000, dg=0x60000, ds=0)
    grad = lambda d, **k: lib.sc_gated_scan_grad(d, *{**base, **k}.values(), 0)  # noqa: E731
    for bad in (dict(dy=0), dict(saved=0), dict(dx=0), dict(dg=0), dict(dx=0x50002), dict(dg=0x50000), dict(dx=0x30000),
                dict(dx=0x40000), dict(dx=0x10000), dict(ds=0x50000), dict(df=0x70002), dict(ds=0x70002),
                dict(df=0x70000, ds=0x70000), dict(dt=-16), dict(saved=0x40002)):
        assert grad(gated(), **bad) == sc.SC_ERR_INVALID, bad
    assert grad(gated(batch=0)) == sc.SC_OK
    step = lambda d, pool=0x50000, rows=2, slots=0, y=0x30000: lib.sc_gated_scan_step(d, pool, rows, slots, y, 16, 0)  # noqa: E731
    one = dict(length=1, x_batch=16, gate_batch=16)
    for bad in (dict(rows=1), dict(pool=0), dict(pool=0x50002), dict(slots=0x60002), dict(y=0x10000), dict(y=0x50000),
                dict(rows=-1), dict(rows=1 << 58), dict(pool=0x10000)):
        assert step(gated(**one), **bad) == sc.SC_ERR_INVALID, bad
    assert step(gated()) == sc.SC_ERR_INVALID  # more than one token
    assert lib.sc_gated_scan_saved_bytes(2, 17, 16) == 2 * 2 * 16 * 4
    assert lib.sc_gated_scan_saved_bytes(2, 0, 16) == lib.sc_gated_scan_saved_bytes(BIG, BIG, 16) == 0


def norm(**k):
    base = dict(dtype=sc.SC_F32, wtype=sc.SC_F32, rms=0, eps=1e-5, batch=2, length=8, channels=16, x=0x10000, x_batch=128,
                x_token=16, residual=0, residual_batch=0, residual_token=0, weight=0x1000, bias=0x2000)
    return seq.NormDesc(**{**base, **k})


def test_norm_refusals(lib):
    base = dict(y=0x20000, yb=128, yt=16, sum=0, sb=0, st=0, saved=0)
    run = lambda d, **k: lib.sc_layer_norm(d, *{**base, **k}.values(), 0)  # noqa: E731
    assert lib.sc_layer_norm(None, 0x20000, 128, 16, 0, 0, 0, 0, 0) == sc.SC_ERR_INVALID
    nan, res = float("nan"), dict(residual=0x30000, residual_batch=128, residual_token=16)
    for bad in (dict(batch=-1), dict(length=-1), dict(channels=-1), dict(x=0), dict(x=0x10002), dict(x_token=-1),
                dict(eps=-1.0), dict(eps=nan), dict(weight=0x1001), dict(bias=0x2002), dict(dtype=10), dict(wtype=-1),
                dict(batch=BIG), dict(length=1 << 31), dict(channels=1 << 31), res):
        assert run(norm(**bad)) == sc.SC_ERR_INVALID, bad
    assert run(norm(dtype=sc.SC_F64)) == sc.SC_ERR_UNSUPPORTED
    assert run(norm(wtype=sc.SC_F16)) == sc.SC_ERR_UNSUPPORTED
    assert run(norm(dtype=sc.SC_F16, wtype=sc.SC_BF16)) == sc.SC_ERR_UNSUPPORTED
    for bad in (dict(y=0), dict(y=0x10000), dict(y=0x1000), dict(yt=15), dict(yb=16), dict(saved=0x40004),
                dict(saved=0x20000), dict(sum=0x30000, sb=128, st=16)):
        assert run(norm(), **bad) == sc.SC_ERR_INVALID, bad
    for bad in (dict(sum=0x30000), dict(sum=0x10000), dict(sum=0x20000), dict(sum=0x40002), dict(sum=0x40000, st=8)):
        assert run(norm(**res), **{**dict(sb=128, st=16), **bad}) == sc.SC_ERR_INVALID, bad
    assert run(norm(batch=0)) == run(norm(channels=0)) == run(norm(length=0)) == sc.SC_OK
    base = dict(dy=0x20000, db=128, dt=16, ds=0, sb=0, st=0, saved=0x40000, dx=0x50000, dw=0, dbias=0)
    grad = lambda d, **k: lib.sc_layer_norm_grad(d, *{**base, **k}.values(), 0)  # noqa: E731
    for bad in (dict(dy=0), dict(saved=0), dict(saved=0x40004), dict(dx=0), dict(dx=0x10000), dict(dx=0x20000),
                dict(dx=0x40000), dict(dw=0x60002), dict(dw=0x50000), dict(dw=0x60000, dbias=0x60000), dict(dw=0x1000),
                dict(ds=0x60002, sb=128, st=16), dict(ds=0x50000, sb=128, st=16), dict(dt=-1)):
        assert grad(norm(), **bad) == sc.SC_ERR_INVALID, bad
    assert grad(norm(channels=0)) == sc.SC_OK
    bytes_ = lib.sc_layer_norm_grad_workspace_bytes
    assert bytes_(2, 8, 16, sc.SC_F32) >= 2 * 16 * 4
    assert bytes_(0, 8, 16, sc.SC_F32) == bytes_(2, 8, 16, sc.SC_I32) == bytes_(1 << 40, 1 << 40, 16, sc.SC_F32) == 0


def test_expert_sort_refusals(lib):
    base = dict(ids=0x10000, ids64=1, entries=8, experts=4, order=0x20000, place=0x30000, offsets=0x40000)
    run = lambda **k: lib.sc_expert_sort(*{**base, **k}.values(), 0)  # noqa: E731
    for bad in (dict(entries=-1), dict(entries=1 << 31), dict(experts=0), dict(experts=-3), dict(ids=0), dict(ids=0x10004),
                dict(order=0), dict(place=0), dict(offsets=0), dict(order=0x20002), dict(offsets=0x40004),
                dict(order=0x10000), dict(place=0x20000), dict(offsets=0x30010)):
        assert run(**bad) == sc.SC_ERR_INVALID, bad
    assert run(experts=1025) == sc.SC_ERR_UNSUPPORTED


def expert(**k):
    base = dict(dtype=sc.SC_F32, wtype=sc.SC_F32, tokens=4, choices=2, dim=8, experts=4, place=0x1000, offsets=0x2000,
                weights=0x3000)
    return seq.ExpertDesc(**{**base, **k})


@pytest.mark.parametrize("name,to_entries", [("sc_expert_gather", True), ("sc_expert_gather_grad", False),
                                             ("sc_expert_combine", False)])
def test_expert_rows_refusals(lib, name, to_entries):
    call = getattr(lib, name)
    run = lambda d, a=0x10000, lda=8, b=0x20000, ldb=8: call(d, a, lda, b, ldb, 0)  # noqa: E731
    assert call(None, 0x10000, 8, 0x20000, 8, 0) == sc.SC_ERR_INVALID
    for bad in (dict(tokens=-1), dict(choices=-1), dict(dim=-1), dict(experts=0), dict(experts=1025), dict(place=0),
                dict(offsets=0), dict(place=0x1002), dict(offsets=0x2004), dict(tokens=1 << 31), dict(choices=1 << 31),
                dict(dtype=-1), dict(dim=BIG)):
        assert run(expert(**bad)) == sc.SC_ERR_INVALID, bad
    assert run(expert(dtype=sc.SC_U32)) == sc.SC_ERR_UNSUPPORTED
    for bad in (dict(lda=7), dict(ldb=7), dict(a=0), dict(b=0), dict(a=0x10002), dict(b=0x10000), dict(b=0x1000),
                dict(b=0x2000)):
        assert run(expert(), **bad) == sc.SC_ERR_INVALID, bad
    if name == "sc_expert_combine":
        assert run(expert(weights=0x3002)) == sc.SC_ERR_INVALID
        assert run(expert(wtype=sc.SC_F16)) == sc.SC_ERR_UNSUPPORTED
        assert run(expert(), b=0x3000) == sc.SC_ERR_INVALID
    assert run(expert(tokens=0)) == run(expert(dim=0)) == sc.SC_OK


def test_expert_combine_grad_refusals(lib):
    base = dict(dout=0x10000, ldo=8, rows=0x20000, ldr=8, drows=0x30000, ldd=8, dw=0x40000)
    run = lambda d, **k: lib.sc_expert_combine_grad(d, *{**base, **k}.values(), 0)  # noqa: E731
    for bad in (dict(dout=0), dict(rows=0), dict(drows=0), dict(ldo=7), dict(ldr=7), dict(ldd=7), dict(dw=0x40002),
                dict(drows=0x20000), dict(drows=0x10000), dict(dw=0x30000), dict(dw=0x3000), dict(dw=0x1000)):
        assert run(expert(), **bad) == sc.SC_ERR_INVALID, bad
    assert run(expert(wtype=sc.SC_I32)) == sc.SC_ERR_UNSUPPORTED
    assert run(expert(tokens=0)) == run(expert(choices=0)) == sc.SC_OK
