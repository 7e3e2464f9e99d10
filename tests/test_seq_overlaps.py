"""Overlaps that the sequence operators refuse: every output against every input and
against every other output, by addresses alone (the checks come before any CUDA call)."""
import itertools

import pytest

import stream_compaction_gb300 as sc
from stream_compaction_gb300 import seq

BATCH, LENGTH, CH, STATES, GROUPS, WIDTH, ROWS = 2, 8, 16, 4, 2, 4, 3
ROW = CH * LENGTH


@pytest.fixture(scope="module")
def lib():
    from stream_compaction_gb300 import build
    build.build()
    return sc.load()


def places(names):
    """An address of its own for every tensor, far apart."""
    return {n: 0x100000 * (i + 1) for i, n in enumerate(names)}


def conv(a, length=LENGTH):
    return seq.ConvDesc(dtype=sc.SC_F32, width=WIDTH, silu=1, reserved=0, batch=BATCH, length=length, channels=CH,
                        x=a["x"], x_batch=CH * length, x_token=CH, weight=a["weight"], bias=a["bias"],
                        heads=a.get("heads", 0), state=a.get("state", 0))


def ssm(a, length=LENGTH):
    bc = GROUPS * STATES
    return seq.SsmDesc(dtype=sc.SC_F32, softplus=1, batch=BATCH, length=length, channels=CH, states=STATES,
                       groups=GROUPS, x=a["x"], dt=a["dt"], x_batch=CH * length, x_token=CH, dt_batch=CH * length,
                       dt_token=CH, A=a["A"], B=a["B"], C=a["C"], B_batch=bc * length, B_token=bc, B_group=STATES,
                       C_batch=bc * length, C_token=bc, C_group=STATES, D=a["D"], z=a["z"], z_batch=CH * length,
                       z_token=CH, dt_bias=a["dt_bias"], heads=a.get("heads", 0), state=a.get("state", 0))


def run_conv(lib, a):
    return lib.sc_causal_conv(conv(a), a["y"], ROW, CH, a["final_state"], 0)


def run_conv_grad(lib, a):
    return lib.sc_causal_conv_grad(conv(a), a["dy"], ROW, CH, a["dx"], ROW, CH, a["dweight"], a["dbias"], a["dstate"], 0)


def run_conv_step(lib, a):
    return lib.sc_causal_conv_step(conv(a, 1), a["pool"], ROWS, a["slots"], a["y"], CH, 0)


def run_scan(lib, a):
    return lib.sc_selective_scan(ssm(a), a["y"], ROW, CH, a["final_state"], a["saved"], 0)


def run_scan_grad(lib, a):
    g = seq.SsmGrads(dy=a["dy"], dy_batch=ROW, dy_token=CH, saved=a["saved"], dfinal=a["dfinal"], dx=a["dx"],
                     ddt=a["ddt"], dz=a["dz"], dB=a["dB"], dC=a["dC"], dA=a["dA"], dD=a["dD"],
                     ddt_bias=a["ddt_bias"], dstate=a["dstate"])
    return lib.sc_selective_scan_grad(ssm(a), g, 0)


def run_scan_step(lib, a):
    return lib.sc_selective_scan_step(ssm(a, 1), a["pool"], ROWS, a["slots"], a["y"], CH, 0)


SSM = ["x", "dt", "A", "B", "C", "D", "z", "dt_bias"]
CALLS = {
    "conv": (run_conv, ["x", "weight", "bias", "heads", "state"], ["y", "final_state"]),
    "conv_grad": (run_conv_grad, ["x", "weight", "bias", "heads", "state", "dy"], ["dx", "dweight", "dbias", "dstate"]),
    "conv_step": (run_conv_step, ["x", "weight", "bias", "slots"], ["y", "pool"]),
    "scan": (run_scan, SSM + ["heads", "state"], ["y", "final_state", "saved"]),
    "scan_grad": (run_scan_grad, SSM + ["heads", "state", "dy", "saved", "dfinal"],
                  ["dx", "ddt", "dz", "dB", "dC", "dA", "dD", "ddt_bias", "dstate"]),
    "scan_step": (run_scan_step, SSM + ["slots"], ["y", "pool"]),
}


@pytest.mark.parametrize("call", CALLS)
def test_an_output_over_an_input_or_another_output(lib, call):
    run, ins, outs = CALLS[call]
    where = places(ins + outs)
    for out, other in itertools.product(outs, ins + outs):
        if out != other:
            assert run(lib, {**where, out: where[other]}) == sc.SC_ERR_INVALID, (out, other)


@pytest.mark.parametrize("call", CALLS)
def test_an_output_that_ends_inside_an_input(lib, call):
    """One row of 16 bytes in common, at the output's end."""
    run, ins, outs = CALLS[call]
    where = places(ins + outs)
    step = call.endswith("step")
    tokens = BATCH * (1 if step else LENGTH)
    size = {"y": tokens * CH, "final_state": BATCH * CH * (STATES if "scan" in call else WIDTH - 1),
            "saved": BATCH * CH * 8, "dx": tokens * CH, "ddt": tokens * CH, "dz": tokens * CH,
            "dB": tokens * GROUPS * STATES, "dC": tokens * GROUPS * STATES, "dA": CH * STATES, "dD": CH, "ddt_bias": CH,
            "dstate": BATCH * CH * (STATES if "scan" in call else WIDTH - 1), "dweight": CH * WIDTH, "dbias": CH,
            "pool": ROWS * CH * (STATES if "scan" in call else WIDTH - 1)}
    for out, other in itertools.product(outs, ins):
        assert run(lib, {**where, out: where[other] - 4 * size[out] + 16}) == sc.SC_ERR_INVALID, (out, other)


def test_empty_calls_still_pass_a_state_on_in_place(lib):
    """No tokens: the state may be its own successor."""
    a = places(["x", "weight", "bias", "y"])
    d = conv(a, 0)
    d.state = 0x900000
    assert lib.sc_causal_conv(d, a["y"], 0, CH, 0x900000, 0) == sc.SC_OK
    a = places(SSM + ["y"])
    d = ssm(a, 0)
    d.state = 0xa00000
    assert lib.sc_selective_scan(d, a["y"], 0, CH, 0xa00000, 0, 0) == sc.SC_OK
