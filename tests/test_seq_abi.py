"""The sequence operators' part of the C ABI: exported symbols, structure sizes, and
the argument checks that return before any CUDA call."""
import ctypes
import os
import re
import subprocess

import pytest

import stream_compaction_gb300 as sc
from stream_compaction_gb300 import seq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from stream_compaction_gb300 import build
    build.build()
    return sc.load()


def test_every_declared_symbol_is_exported_and_bound(lib):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "sc_seq.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(sc_[a-z_0-9]+)\s*\(", src))
    assert names == set(seq.SIGNATURES)
    out = subprocess.run(["nm", "-D", "--defined-only", sc.LIB_PATH], capture_output=True, text=True).stdout
    assert names <= set(re.findall(r" T (sc_\w+)", out))


def test_structures_match_the_header(tmp_path):
    """Sizes and last offsets of the ctypes structures against the C compiler's."""
    src = tmp_path / "s.c"
    src.write_text('#include "sc_seq.h"\n#include <stdio.h>\nint main(void) { printf("%zu %zu %zu %zu %zu %zu\\n", '
                   'sizeof(sc_conv_desc), sizeof(sc_ssm_desc), sizeof(sc_ssm_grads), offsetof(sc_conv_desc, state), '
                   'offsetof(sc_ssm_desc, state), offsetof(sc_ssm_grads, dstate)); return 0; }\n')
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-I" + os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(seq.ConvDesc), ctypes.sizeof(seq.SsmDesc), ctypes.sizeof(seq.SsmGrads),
                   seq.ConvDesc.state.offset, seq.SsmDesc.state.offset, seq.SsmGrads.dstate.offset]


def embed(lib, ids=0x1000, ids64=1, tokens=4, dtype=sc.SC_F32, weight=0x10000, vocab=10, dim=8, ldw=8, out=0x20000,
          ldo=8):
    return lib.sc_embed(ids, ids64, tokens, dtype, weight, vocab, dim, ldw, 1.0, out, ldo, 0)


def test_embed_refusals(lib):
    assert embed(lib, tokens=-1) == sc.SC_ERR_INVALID
    assert embed(lib, tokens=1 << 31) == sc.SC_ERR_INVALID
    assert embed(lib, vocab=1 << 31) == sc.SC_ERR_INVALID
    assert embed(lib, dtype=11) == sc.SC_ERR_INVALID
    assert embed(lib, dtype=sc.SC_I32) == sc.SC_ERR_UNSUPPORTED
    assert embed(lib, ldw=7) == sc.SC_ERR_INVALID
    assert embed(lib, ids=0) == sc.SC_ERR_INVALID
    assert embed(lib, ids=0x1004) == sc.SC_ERR_INVALID          # int64 ids on 4 bytes
    assert embed(lib, out=0x10010) == sc.SC_ERR_INVALID         # inside the weight
    assert embed(lib, weight=0x10002) == sc.SC_ERR_INVALID
    assert embed(lib, tokens=0, ids=0, weight=0, out=0) == sc.SC_OK
    grad = lambda **k: lib.sc_embed_grad(*[{**dict(ids=0x1000, ids64=1, tokens=4, dtype=sc.SC_BF16, dout=0x10000, ldd=8,  # noqa: E731
                                                   vocab=10, dim=8, scale=1.0, wtype=sc.SC_BF16, dw=0x20000, ldw=8,
                                                   acc=0, s=0), **k}[n] for n in
                                           ("ids", "ids64", "tokens", "dtype", "dout", "ldd", "vocab", "dim", "scale",
                                            "wtype", "dw", "ldw", "acc", "s")])
    assert grad(wtype=sc.SC_F16) == sc.SC_ERR_UNSUPPORTED
    assert grad(ldd=4) == sc.SC_ERR_INVALID
    assert grad(dw=0) == sc.SC_ERR_INVALID
    assert grad(dw=0x10000) == sc.SC_ERR_INVALID
    assert grad(vocab=0) == sc.SC_OK
    assert lib.sc_embed_grad_workspace_bytes(-1, 5, 5) == 0
    assert lib.sc_embed_grad_workspace_bytes(1000, 50000, 64) >= 4 * 4 * 1000


def conv(**k):
    base = dict(dtype=sc.SC_F32, width=4, silu=1, reserved=0, batch=2, length=8, channels=16, x=0x10000, x_batch=128,
                x_token=16, weight=0x1000, bias=0, heads=0, state=0)
    return seq.ConvDesc(**{**base, **k})


def test_conv_refusals(lib):
    run = lambda d, y=0x20000, yb=128, yt=16, fs=0: lib.sc_causal_conv(d, y, yb, yt, fs, 0)  # noqa: E731
    assert lib.sc_causal_conv(None, 0x20000, 128, 16, 0, 0) == sc.SC_ERR_INVALID
    for bad in (dict(width=0), dict(width=9), dict(batch=-1), dict(length=-1), dict(channels=-3), dict(x=0),
                dict(x=0x10001), dict(weight=0), dict(x_token=-1), dict(reserved=1), dict(dtype=12),
                dict(batch=1 << 40)):
        assert run(conv(**bad)) == sc.SC_ERR_INVALID, bad
    assert run(conv(dtype=sc.SC_I64)) == sc.SC_ERR_UNSUPPORTED
    assert run(conv(), y=0x10040) == sc.SC_ERR_INVALID            # shares rows of x
    assert run(conv(), yt=8) == sc.SC_ERR_INVALID                 # rows of y on one another
    assert run(conv(), yb=64) == sc.SC_ERR_INVALID
    assert run(conv(state=0x30000), fs=0x30000) == sc.SC_ERR_INVALID
    assert run(conv(batch=0)) == sc.SC_OK
    assert run(conv(channels=0)) == sc.SC_OK
    g = lib.sc_causal_conv_grad
    assert g(conv(), 0, 128, 16, 0x40000, 128, 16, 0, 0, 0, 0) == sc.SC_ERR_INVALID
    assert g(conv(), 0x20000, 128, 16, 0x20000, 128, 16, 0, 0, 0, 0) == sc.SC_ERR_INVALID
    assert g(conv(), 0x20000, 128, 16, 0x40000, 128, 16, 0x50002, 0, 0, 0) == sc.SC_ERR_INVALID
    step = lambda d, pool=0x50000, rows=2, slots=0, y=0x20000: lib.sc_causal_conv_step(d, pool, rows, slots, y, 16, 0)  # noqa: E731
    one = dict(length=1, x_batch=16)
    assert step(conv(**one), rows=1) == sc.SC_ERR_INVALID         # fewer rows than the batch, no slots
    assert step(conv(), rows=2) == sc.SC_ERR_INVALID              # more than one token
    assert step(conv(**one), pool=0) == sc.SC_ERR_INVALID
    assert step(conv(**one), y=0x10000) == sc.SC_ERR_INVALID
    assert step(conv(**one), y=0x50000) == sc.SC_ERR_INVALID


def ssm(**k):
    base = dict(dtype=sc.SC_F32, softplus=1, batch=2, length=8, channels=16, states=4, groups=1, x=0x10000, dt=0x20000,
                x_batch=128, x_token=16, dt_batch=128, dt_token=16, A=0x1000, B=0x30000, C=0x40000, B_batch=32,
                B_token=4, B_group=4, C_batch=32, C_token=4, C_group=4, D=0, z=0, z_batch=0, z_token=0, dt_bias=0,
                heads=0, state=0)
    return seq.SsmDesc(**{**base, **k})


def test_scan_refusals(lib):
    run = lambda d, y=0x50000, fs=0, saved=0, yt=16: lib.sc_selective_scan(d, y, 128, yt, fs, saved, 0)  # noqa: E731
    assert lib.sc_selective_scan(None, 0x50000, 128, 16, 0, 0, 0) == sc.SC_ERR_INVALID
    for bad in (dict(states=0), dict(groups=0), dict(groups=3), dict(batch=-1), dict(length=-1), dict(x=0), dict(dt=0),
                dict(A=0), dict(B=0), dict(C=0x40001), dict(z=0x60001), dict(D=0x1002), dict(x_token=-16),
                dict(dtype=-1), dict(length=1 << 50)):
        assert run(ssm(**bad)) == sc.SC_ERR_INVALID, bad
    assert run(ssm(states=65)) == sc.SC_ERR_UNSUPPORTED
    assert run(ssm(dtype=sc.SC_U32)) == sc.SC_ERR_UNSUPPORTED
    assert run(ssm(), y=0x10000) == sc.SC_ERR_INVALID
    assert run(ssm(), yt=15) == sc.SC_ERR_INVALID
    assert run(ssm(), saved=0x60004) == sc.SC_ERR_INVALID
    assert run(ssm(state=0x70000), fs=0x70000) == sc.SC_ERR_INVALID
    assert run(ssm(batch=0)) == sc.SC_OK
    grads = dict(dy=0x60000, dy_batch=128, dy_token=16, saved=0x70000, dfinal=0, dx=0x80000, ddt=0x90000, dz=0,
                 dB=0xa0000, dC=0xb0000, dA=0xc0000, dD=0, ddt_bias=0, dstate=0)
    g = lambda d, **k: lib.sc_selective_scan_grad(d, seq.SsmGrads(**{**grads, **k}), 0)  # noqa: E731
    for bad in (dict(dy=0), dict(saved=0), dict(dx=0), dict(ddt=0), dict(dA=0), dict(dB=0), dict(dz=0xd0000),
                dict(dx=0x10000), dict(ddt=0x80000), dict(dC=0xa0000)):
        assert g(ssm(), **bad) == sc.SC_ERR_INVALID, bad
    assert g(ssm(z=0xe0000, z_batch=128, z_token=16)) == sc.SC_ERR_INVALID  # dz is missing
    step = lambda d, pool=0x80000, rows=2, y=0x50000: lib.sc_selective_scan_step(d, pool, rows, 0, y, 16, 0)  # noqa: E731
    one = dict(length=1, x_batch=16, dt_batch=16, B_batch=4, C_batch=4)
    assert step(ssm(**one), rows=1) == sc.SC_ERR_INVALID
    assert step(ssm()) == sc.SC_ERR_INVALID
    assert step(ssm(**one), pool=0x80002) == sc.SC_ERR_INVALID
    assert step(ssm(**one), y=0x20000) == sc.SC_ERR_INVALID
    assert lib.sc_selective_scan_saved_bytes(2, 17, 16, 4) == 2 * 2 * 16 * 8 * 4
    assert lib.sc_selective_scan_saved_bytes(2, 17, 16, 65) == 0
    assert lib.sc_selective_scan_grad_workspace_bytes(2, 17, 16, 4, 3) == 0


def test_column_slices_of_a_joint_buffer_do_not_overlap(lib):
    # x and y as the two halves of rows of 32: same strides, disjoint columns; one column over is refused
    halves = conv(length=0, x_batch=256, x_token=32)
    assert lib.sc_causal_conv(halves, 0x10040, 256, 32, 0, 0) == sc.SC_OK  # no tokens: nothing runs
    assert lib.sc_causal_conv(conv(x_batch=256, x_token=32), 0x1003c, 256, 32, 0, 0) == sc.SC_ERR_INVALID
